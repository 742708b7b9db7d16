// Attention with many rows a sequence (prefill chunks) on the tensor cores.
//
// A CTA holds NRT row tiles of 128 rows (new token, query head of the kv
// head's group) and walks the keys 64 at a time:
//   loader (1 warp)     bulk copies of the pool's half tiles (32 keys' K or V
//                       with their scales) into two rings
//   dequantise (4 + 4)  integer times scale, rounded to fp16 once, into
//                       128-byte swizzled stages: four warps K as the K-major,
//                       four V, which has the same rows, as the MN-major operand
//   issue (1 a tile)    S = Q K^T (tcgen05.mma, fp32 in tensor memory, two
//                       buffers a row tile), O += P V with P read from tensor
//                       memory, and so is Q where it fits (heads of 64 and 256):
//                       products of 64 keys with both operands in shared
//                       memory take 48 cycles, with Q in tensor memory 32
//   softmax (4 a tile)  a thread a row: maximum, exponentials, sum; P goes
//                       back into S's columns as fp16 (times 2^8, as in
//                       attend_rows_kernel).  O is rescaled in tensor memory
//                       only when a maximum grew by more than 2^7 since the
//                       last time, which keeps P below fp16's largest.
// An fp16 K has 11 bits where integer times scale has up to 19.  That is
// within what outputs of bf16 show; with fp16 activations it was the largest
// error (5.4e-4 of the output, of 2.1e-4 for its own rounding), so there the
// rest of K, exact in fp16 too, is a second operand of S, and P's of O.
// Registers move from the dequantising warps to the softmax (setmaxnreg).
// The two row tiles share the dequantised keys and keep the tensor core busy
// while the other's softmax runs.  A step of 64 keys (heads of 128, 256 rows)
// is 24 products, 1,240 cycles of the tensor core; one warp that issued both
// tiles' products, with its waits and elections, took 2,500.  2,048 new tokens
// of 8,192 (32 query and 4 kv heads of 128, 8 bits, bf16) take 230 us (1,046
// TFLOP/s), 8,192 of 16,384 1,350 (1,220); the chain of a step's softmax bounds them.
//
// The line of work is measured in keys, causal limits included, so that all
// parts cost the same: row tile rt of a sequence costs kSegmentKeys + the keys
// in front of its new tokens + (rt + 1) * rows / group, in units of 1 / group.
//
// 4-bit elements leave the dequantisation in the order 0 4 1 5 2 6 3 7 within
// each eight; queries are stored in the same order, and the output's is undone
// when it is written.
#pragma once

#include "moe_attend.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kKeys = 64;           // keys of a step
constexpr int kSegmentKeys = 768;   // what a segment costs beside its keys, in keys
constexpr float kGrow = 7.f;        // log2 by which a maximum may outgrow its reference
constexpr int kDeqWarps = 4;        // of either stream

template <int D, int BITS, bool BF16>
struct TilesPlan {
  static constexpr int NRT = D == 256 ? 1 : 2;
  static constexpr int kRows = 128 * NRT;
  static constexpr int kHalf = kv_half_bytes(D, BITS);
  static constexpr bool kRest = !BF16;                           // K's and P's rests, too
  static constexpr int kHalves = D == 256 && (BITS == 8 || kRest) ? 1 : 2;  // half tiles of a ring entry
  static constexpr int kEntry = kHalves * kHalf;
  static constexpr int kEntries = D == 256 ? (kRest ? (BITS == 8 ? 2 : 3) : 4) : 3;  // of either ring
  static constexpr int kStage = kKeys * D * 2, kKStage = kStage * (kRest ? 2 : 1);
  static constexpr bool kQTmem = D != 128;  // queries in tensor memory
  static constexpr int kQ = kQTmem ? 0 : 128 * D * 2;
  static constexpr int kOffK = NRT * kQ;
  static constexpr int kOffV = kOffK + 2 * kKStage;
  static constexpr int kOffRaw = kOffV + 2 * kStage;
  static constexpr int kOffBar = (kOffRaw + 2 * kEntries * kEntry + 15) & ~15;
  // barriers: raw full and empty of either ring, K full and empty, V full and empty, Q full, S full, P full, O done, pieces done
  static constexpr int kSlots = 8;  // pieces under way at most
  static constexpr int kBars = 4 * kEntries + 8 + NRT * 6 + kSlots;
  static constexpr int kOffMisc = kOffBar + 8 * kBars;
  static constexpr int kSoftWarps = 4 * NRT;
  static constexpr int kThreads = 32 * (kSoftWarps + 2 * kDeqWarps + 4);
  static constexpr int kSmem = kOffMisc + 72 + kThreads / 32 * 8;
  // registers of the roles' warpgroups: together no more than the launch's
  static constexpr int kLaunchRegs = NRT == 2 ? 96 : 128;
  static constexpr int kSoftRegs = NRT == 2 ? 152 : 208, kDeqRegs = NRT == 2 ? 64 : 104, kRestRegs = NRT == 2 ? 48 : 96;
  static_assert(kSoftWarps * kSoftRegs + 2 * kDeqWarps * kDeqRegs + 4 * kRestRegs <= kThreads / 32 * kLaunchRegs, "registers");
  static constexpr int kTmemO = NRT * 2 * kKeys;  // S buffers first, then O
  static constexpr int kTmemQ = kTmemO + NRT * D;
  static constexpr int kTmemCols = 512;
  static_assert(kSmem <= 232448, "shared memory of an SM");
  static_assert(kTmemQ + (kQTmem ? NRT * D / 2 : 0) <= kTmemCols, "tensor memory");
};

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Four products, K = 64, the first adding to D if acc.  The whole warp calls
// these with the same operands and one lane issues: under a branch of one
// lane the operands' way into uniform registers costs more than the product
// does, and so does an election for each.
__device__ __forceinline__ void tc_mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, %3, %3;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory: two fp16 of a row in each 32-bit column.  B advances by B_STEP 16-byte units.
template <int B_STEP>
__device__ __forceinline__ void tc_mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, t, e;\n .reg .b32 a;\n .reg .b64 b;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, %3, %3;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n add.s32 a, %1, 8;\n add.s64 b, %2, %5;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n add.s32 a, %1, 16;\n add.s64 b, %2, 2 * %5;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n add.s32 a, %1, 24;\n add.s64 b, %2, 3 * %5;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "n"(B_STEP)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand descriptors, 128-byte swizzle.  K-major: rows of 64
// fp16, 8-row atoms 1,024 B apart.  MN-major: the same bytes with the 64 fp16
// along N, K groups of 8 rows 1,024 B apart and the next 64 of N a panel away.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t panel) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16: D fp32, A and B fp16, M = 128, N; B MN-major when asked.
__device__ __forceinline__ constexpr uint32_t instr_desc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// A part of a segment: key steps t0 .. t1 of row tile rt.
struct Piece {
  int b, head, rt, t0, t1, steps;
  int rows;        // live rows of the row tile
  int first_part;  // the CTA that has step 0
  int lim;         // keys that hold anything
  Seq sq;
};

// a / b of numbers >= 0, mostly of 31 bits, when a shorter division does: 2,048
// new tokens of 8,192 take 230 us with it and 242 without.  Not with row tiles
// of 128 (heads of 256), where the kernel comes out slower for it in every case
// measured, of unknown cause: 12 sequences of 60,000 to 131,072 tokens in 4
// bits 219 us without and 250 with it, 16 of 16,384 with 24 rows each 71 and 83, in
// 8 bits 81 and 89.
template <int ROWS>
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ROWS == 256 && ((a | b) >> 31) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The CTA's share of the line of work.  With a shared prefix there is one
// sequence, `pre`: the new tokens of all, in front of them as many keys as the
// prefix has (its len), read through the block table's row b.
template <int ROWS>
struct Walk {
  long long part, w1, cur, base;
  int b;
  Seq pre;

  // Cost of a head's row tiles 0 .. rt - 1, in keys times the group.
  static __device__ __forceinline__ long long cost(const AttArgs& t, const Seq& s, long long rt) {
    if (t.shared) return rt * t.group * (kSegmentKeys + (long long)s.len);
    return rt * t.group * (kSegmentKeys + (long long)max(s.len - s.n, 0)) + (long long)ROWS * rt * (rt + 1) / 2;
  }
  static __device__ __forceinline__ int row_tiles(const AttArgs& t, const Seq& s) { return (s.n * t.group + ROWS - 1) / ROWS; }

  __device__ bool next(const KvArgs& a, const AttArgs& t, Piece& p) {
    while (cur < w1) {
      const Seq s = t.shared ? pre : seq_at(a, b);
      const int n_rt = row_tiles(t, s);
      const long long per_head = cost(t, s, n_rt), local = cur - base;
      if (local >= per_head * a.heads) {
        base += per_head * a.heads;
        ++b;
        continue;
      }
      const int head = (int)quotient<ROWS>(local, per_head);
      const long long x = local - head * per_head;
      int lo = 0, hi = n_rt - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost(t, s, mid) <= x)
          lo = mid;
        else
          hi = mid - 1;
      }
      const long long c0 = cost(t, s, lo), all = cost(t, s, lo + 1) - c0;
      const long long x0 = x - c0, x1 = min(all, x0 + (w1 - cur)), seg_start = cur - x0;
      cur += x1 - x0;
      // the keys that the tile's last row sees
      const int last = min((lo + 1) * ROWS, s.n * t.group) - 1;
      p.lim = min(s.len, a.max_pages * a.page_size);
      const int lim = t.shared ? p.lim : min(s.len - s.n + last / t.group + 1, p.lim);
      p.steps = lim > 0 ? (lim - 1) / kKeys + 1 : 1;
      auto step_at = [&](long long pos) {
        const long long u = quotient<ROWS>(pos, t.group) - kSegmentKeys;
        return (int)min((long long)p.steps, (max(u, 0ll) + kKeys - 1) / kKeys);
      };
      p.t0 = step_at(x0);
      p.t1 = x1 == all ? p.steps : step_at(x1);
      if (p.t1 <= p.t0) continue;
      p.b = b;
      p.head = head;
      p.rt = lo;
      p.rows = s.n * t.group - lo * ROWS;
      p.sq = s;
      p.first_part = (int)quotient<ROWS>(seg_start + min((long long)t.group * (kSegmentKeys + 1), all) - 1, part);
      return true;
    }
    return false;
  }
};

// The integers times scales of an entry's HALVES * 32 keys into rows key_base
// .. of a stage, all loads first.  V: keys from lim on (of the first key) are
// seen by no row and become 0, and so do blocks of non-finite scale; the
// first such key's position goes to `bad`.  REST, K: what the rounding left
// goes a stage further.
template <int D, int BITS, int HALVES, bool REST>
__device__ __forceinline__ void dequantise(uint32_t raw, uint32_t stage, int key_base, int tid, bool is_v, int lim, int pos0, int* bad,
                                           uint32_t magic) {
  constexpr int R = kv_row_bytes(D, BITS), UPR = R / 16, EPU = 128 / BITS;  // 16-byte units a row, elements a unit
  constexpr int N = (UPR + kDeqWarps - 1) / kDeqWarps;                      // units a thread and half
  const int key = tid & 31, turn = kv_turn(key) & (UPR - 1);
  uint4 w4[HALVES][N];
  uint32_t s2[HALVES][N];
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = n * kDeqWarps + (tid >> 5);
      if (UPR < kDeqWarps && c >= UPR) break;
      const uint32_t at = raw + h * kv_half_bytes(D, BITS);
      w4[h][n] = lds128(at + key * R + ((c ^ turn) << 4));
      s2[h][n] = lds16(at + kKvTile * R + ((c * EPU / 32) * kKvTile + key) * 2);
    }
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    const int k = h * 32 + key, row = key_base + k;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = n * kDeqWarps + (tid >> 5);
      if (UPR < kDeqWarps && c >= UPR) break;
      uint32_t sc = s2[h][n];
      if (is_v) {
        if (k >= lim) {
          sc = 0;
        } else if ((sc & 0x7C00u) == 0x7C00u) {
          sc = 0;
          atomicMin(bad, pos0 + k);
        }
      }
      sc = prmt(sc, sc, 0x1010);
      const uint32_t w[4] = {w4[h][n].x, w4[h][n].y, w4[h][n].z, w4[h][n].w};
#pragma unroll
      for (int i = 0; i < EPU / 8; ++i) {
        uint32_t x[4];  // the integers
        if (BITS == 8) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            x[2 * j] = hsub2(prmt(w[2 * i + j], magic, 0x5150), 0x64806480u);
            x[2 * j + 1] = hsub2(prmt(w[2 * i + j], magic, 0x5352), 0x64806480u);
          }
        } else {
          const uint32_t v = w[i], v8 = v >> 8;
          x[0] = hsub2(and_or<0x000F000Fu>(v, magic), 0x64086408u);
          x[1] = hfma2(and_or<0x00F000F0u>(v, magic), 0x2C002C00u, 0xD480D480u);
          x[2] = hsub2(and_or<0x000F000Fu>(v8, magic), 0x64086408u);
          x[3] = hfma2(and_or<0x00F000F0u>(v8, magic), 0x2C002C00u, 0xD480D480u);
        }
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = hmul2(x[j], sc);
        const int oc = c * (EPU / 8) + i;  // chunk of 8 elements
        const uint32_t to = stage + (oc >> 3) * (kKeys * 128) + row * 128 + (((oc & 7) ^ (row & 7)) << 4);
        sts128(to, y[0], y[1], y[2], y[3]);
        if (REST && !is_v) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = hfma2(x[j], sc, y[j] ^ 0x80008000u);
          sts128(to + kKeys * D * 2, x[0], x[1], x[2], x[3]);
        }
      }
    }
  }
}

template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, int BITS, bool BF16>
__global__ void __launch_bounds__((TilesPlan<D, BITS, BF16>::kThreads), 1) attend_tiles_kernel(const KvArgs a, const AttArgs t) {
  using P = TilesPlan<D, BITS, BF16>;
  constexpr int NRT = P::NRT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sm = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [&](int i) { return sm + P::kOffBar + 8 * i; };
  constexpr int kRawFull = 0, kRawEmpty = 2 * P::kEntries, kKFull = 4 * P::kEntries,  // raw: K's ring, then V's
                kKEmpty = kKFull + 2, kVFull = kKEmpty + 2,
                kVEmpty = kVFull + 2, kQFull = kVEmpty + 2, kSFull = kQFull + NRT, kPFull = kSFull + 2 * NRT,
                kODone = kPFull + 2 * NRT, kPieceDone = kODone + NRT;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + P::kOffMisc);
  // by piece: position of the first bad page or non-finite V.  The loader clears a slot before it loads the piece, when all
  // softmax warps are done with the slot's last one (kPieceDone)
  int* s_bad = reinterpret_cast<int*>(smem + P::kOffMisc + 16);
  int& s_b = *reinterpret_cast<int*>(smem + P::kOffMisc + 48);
  int* s_long = reinterpret_cast<int*>(smem + P::kOffMisc + 52);  // [2]
  long long& s_base = *reinterpret_cast<long long*>(smem + P::kOffMisc + 64);
  long long* s_sum = reinterpret_cast<long long*>(smem + P::kOffMisc + 72);  // [warps]

  if (tid == 0) {
    for (int i = 0; i < 2 * P::kEntries; ++i) {
      mbar_init(bar(kRawFull + i), 1);
      mbar_init(bar(kRawEmpty + i), kDeqWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kKFull + i), kDeqWarps);
      mbar_init(bar(kKEmpty + i), NRT);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kVFull + i), kDeqWarps);
      mbar_init(bar(kVEmpty + i), NRT);
    }
    for (int i = 0; i < NRT; ++i) {
      mbar_init(bar(kQFull + i), 4);
      for (int j = 0; j < 2; ++j) {
        mbar_init(bar(kSFull + 2 * i + j), 1);
        mbar_init(bar(kPFull + 2 * i + j), 4);
      }
      mbar_init(bar(kODone + i), 1);
    }
    for (int i = 0; i < P::kSlots; ++i) mbar_init(bar(kPieceDone + i), P::kSoftWarps);
    fence_mbar_init();
  }
  auto bad_of = [&](int piece) { return &s_bad[piece % P::kSlots]; };
  // the slot's last piece has been finished by all
  auto slot_wait = [&](int piece, bool& ok) { mbar_wait(bar(kPieceDone + piece % P::kSlots), ((piece / P::kSlots) & 1) ^ 1, ok); };
  constexpr int kIssueWarp = P::kSoftWarps + 2 * kDeqWarps, kLoadWarp = kIssueWarp + 1;  // (the second row tile's products: kIssueWarp + 2)
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)), "n"(P::kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }

  // the line of work: each thread sums its share of the sequences
  using W = Walk<P::kRows>;
  const int chunk = (a.n_seqs + P::kThreads - 1) / P::kThreads;
  const int b_lo = min(tid * chunk, a.n_seqs), b_hi = min(b_lo + chunk, a.n_seqs);
  long long mine = 0;
  int longest = 0, longest_b = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = seq_at(a, b);
    mine += W::cost(t, s, W::row_tiles(t, s)) * a.heads;
    if (s.len > longest) longest = s.len, longest_b = b;
    if (blockIdx.x == 0) flag_batch(a, b);
  }
  if (t.shared) {  // the prefix is read through the longest sequence's row; there are no keys behind that one's length
    if (tid == 0) s_long[0] = s_long[1] = 0;
    __syncthreads();
    atomicMax(&s_long[0], longest);
    __syncthreads();
    if (longest > 0 && longest == s_long[0]) s_long[1] = longest_b;  // (any of them)
    mine = 0;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  tc_before();
  __syncthreads();
  tc_after();
  long long total = 0, before = incl - mine;
  for (int w = 0; w < P::kThreads / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  W walk;
  // a part spans two steps at least, so that none between a segment's first and last is empty
  if (t.shared) {
    const int n = min(max(__ldg(a.cu + a.n_seqs), 0), a.n_tokens);
    walk.pre = Seq{0, n, min(t.shared, s_long[0]), false};
    total = n > 0 && walk.pre.len > 0 ? W::cost(t, walk.pre, W::row_tiles(t, walk.pre)) * a.heads : 0;
  }
  walk.part = max(quotient<P::kRows>(total + gridDim.x - 1, gridDim.x), (long long)t.group * 2 * kKeys);
  walk.cur = (long long)blockIdx.x * walk.part;
  walk.w1 = min(walk.cur + walk.part, total);
  if (t.shared) {
    if (tid == 0) s_base = 0, s_b = s_long[1];
  } else if (walk.cur < total && before <= walk.cur && walk.cur < before + mine) {
    s_base = before;
    s_b = b_lo;
  }
  if (tid == 0) t.ends[blockIdx.x].first = -1;
  __syncthreads();
  grid_launch_dependents();
  walk.base = s_base;
  walk.b = s_b;
  const uint32_t tmem = *s_tmem;
  bool ok = true;
  Piece p;

  if (warp >= kIssueWarp) {
    give_registers<P::kRestRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- loader
      int entry = 0, piece = 0;
      uint32_t phase = 1;  // the ring starts empty
      for (; walk.next(a, t, p); ++piece) {
        slot_wait(piece, ok);
        if (lane == 0) *bad_of(piece) = INT32_MAX;
        __syncwarp();
        const int lim = p.lim;
        const int n32 = 2 * (p.t1 - p.t0);
        const uint8_t* src = nullptr;
        for (int i = 0; i < n32; ++i) {
          if ((i & 31) == 0) {  // lane j looks up the page of the tile i + j
            const int pos = (2 * p.t0 + i + lane) * kKvTile;
            int page = 0, pi = 0;
            if (i + lane < n32 && pos < lim) {
              pi = kv_page_of(a, pos);
              page = __ldg(a.table + (size_t)p.b * a.table_stride + pi);
              if ((unsigned)page >= (unsigned)a.n_pages) {
                atomicMin(bad_of(piece), pos);
                kv_flag(a, MOE_KV_BAD_PAGE);
                page = 0;  // in bounds; the rows that see it become NaN
              }
            }
            const int in_page = pos < lim ? pos - pi * a.page_size : 0;  // (behind the last key: any tile, nothing of it is seen)
            src = a.data + (size_t)page * a.page_bytes + (size_t)p.head * a.head_bytes + (size_t)(in_page / kKvTile) * (2 * P::kHalf);
          }
          // the tiles of an entry, K then V; the lane that looked a tile up copies it
          if (i % P::kHalves) continue;
          for (int v = 0; v < 2; ++v) {
            const int e = v * P::kEntries + entry;
            mbar_wait(bar(kRawEmpty + e), phase, ok);
            if (lane == 0 && ok) mbar_expect_tx(bar(kRawFull + e), P::kEntry);  // (who has not seen the entry given back does not fill it)
            __syncwarp();
            if (ok && lane >= (i & 31) && lane < (i & 31) + P::kHalves)
              bulk_g2s(sm + P::kOffRaw + e * P::kEntry + (lane - (i & 31)) * P::kHalf, src + v * P::kHalf, P::kHalf, bar(kRawFull + e));
          }
          if (++entry == P::kEntries) entry = 0, phase ^= 1;
        }
      }
    } else if (warp == kIssueWarp || (NRT == 2 && warp == kIssueWarp + 2)) {
      // ---------------------------------------------------------------- issue, a warp a row tile
      constexpr uint32_t kIdS = instr_desc(kKeys, false), kIdO = instr_desc(D, true);
      const int i = warp == kIssueWarp ? 0 : 1;
      uint32_t step = 0, own = 0, pieces = 0;  // steps over all pieces; the row tile's steps and pieces
      while (walk.next(a, t, p)) {
        const int n = p.t1 - p.t0;
        if (i * 128 >= p.rows) {  // no rows in the tile: the stages pass by
          for (int j = 0; j < n; ++j, ++step) {
            mbar_wait(bar(kKFull + (step & 1)), (step >> 1) & 1, ok);
            if (lane == 0) mbar_arrive(bar(kKEmpty + (step & 1)));
            mbar_wait(bar(kVFull + (step & 1)), (step >> 1) & 1, ok);
            if (lane == 0) mbar_arrive(bar(kVEmpty + (step & 1)));
          }
          continue;
        }
        mbar_wait(bar(kQFull + i), pieces++ & 1, ok);
        for (int j = 0; j <= n; ++j) {
          if (j < n) {
            const uint32_t st = (step + j) & 1, sb = (own + j) & 1;
            const uint32_t k = sm + P::kOffK + st * P::kKStage, d = tmem + (2 * i + sb) * kKeys;
            mbar_wait(bar(kKFull + st), ((step + j) >> 1) & 1, ok);
            tc_after();
#pragma unroll
            for (int x = 0; x < D / 64 * (P::kRest ? 2 : 1); ++x) {  // (the rest lies a stage, D / 64 panels, further)
              const uint64_t kd = desc_k(k + x * (kKeys * 128));
              const int panel = x % (D / 64);
              if (P::kQTmem)
                tc_mma4_ts<2>(d, tmem + P::kTmemQ + i * (D / 2) + panel * 32, kd, kIdS, x > 0);
              else
                tc_mma4(d, desc_k(sm + i * P::kQ + panel * (128 * 128)), kd, kIdS, x > 0);
            }
            tc_commit(bar(kSFull + 2 * i + sb));
            tc_commit(bar(kKEmpty + st));
          }
          if (j > 0) {
            const uint32_t f = step + j - 1, st = f & 1, of = own + j - 1, pb = of & 1;
            mbar_wait(bar(kVFull + st), (f >> 1) & 1, ok);
            mbar_wait(bar(kPFull + 2 * i + pb), (of >> 1) & 1, ok);
            tc_after();
            static_assert(kKeys == 64, "one call");
            const uint32_t from = tmem + (2 * i + pb) * kKeys, o = tmem + P::kTmemO + i * D;
            const uint64_t vd = desc_mn(sm + P::kOffV + st * P::kStage, kKeys * 128);
            tc_mma4_ts<2048 / 16>(o, from, vd, kIdO, j > 1);
            if (P::kRest) tc_mma4_ts<2048 / 16>(o, from + kKeys / 2, vd, kIdO, 1);
            tc_commit(bar(kODone + i));
            tc_commit(bar(kVEmpty + st));
          }
        }
        step += n;
        own += n;
      }
    }
  } else if (warp >= P::kSoftWarps) {
    // ---------------------------------------------------------------- dequantise
    give_registers<P::kDeqRegs>();
    const int dt = tid & 127;
    const bool v = warp >= P::kSoftWarps + kDeqWarps;  // which stream
    uint32_t magic = 0x64006400u;
    asm volatile("" : "+r"(magic));
    int entry = 0;
    uint32_t phase = 0, step = 0;
    for (int piece = 0; walk.next(a, t, p); ++piece) {
      const int lim = p.lim;
      for (int j = p.t0; j < p.t1; ++j, ++step) {
        const uint32_t st = step & 1;
        mbar_wait(v ? bar(kVEmpty + st) : bar(kKEmpty + st), ((step >> 1) & 1) ^ 1, ok);
#pragma unroll
        for (int h = 0; h < 2; h += P::kHalves) {
          const int pos0 = j * kKeys + h * kKvTile, e = (v ? P::kEntries : 0) + entry;
          mbar_wait(bar(kRawFull + e), phase, ok);
          dequantise<D, BITS, P::kHalves, P::kRest>(sm + P::kOffRaw + e * P::kEntry,
                                                    sm + (v ? P::kOffV + st * P::kStage : P::kOffK + st * P::kKStage), h * kKvTile, dt, v,
                                                    lim - pos0, pos0, bad_of(piece), magic);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kRawEmpty + e));
          if (++entry == P::kEntries) entry = 0, phase ^= 1;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(v ? bar(kVFull + st) : bar(kKFull + st));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    take_registers<P::kSoftRegs>();
    const int i = warp >> 2, row = tid & 127;  // row tile, row in it
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t t_o = tmem + P::kTmemO + i * D + lanes;
    uint32_t step = 0;
    for (int piece = 0; walk.next(a, t, p); ++piece) {
      auto finished = [&]() {
        if (lane == 0) mbar_arrive(bar(kPieceDone + piece % P::kSlots));
      };
      if (i * 128 >= p.rows) {  // no rows in this tile
        slot_wait(piece, ok);   // (nothing else holds the warp back)
        finished();
        continue;
      }
      const int fr = p.rt * P::kRows + i * 128 + row, tok = fr / t.group, gh = fr - tok * t.group;
      bool live = fr < p.sq.n * t.group;
      int see = live ? p.sq.len - p.sq.n + tok : -1;  // the last position that the row sees
      if (t.shared && live) {
        const int b = kv_seq_of(a, tok);
        const Seq own = seq_at(a, max(b, 0));
        live = b >= 0 && tok - own.row0 < own.n;
        see = live ? min(own.len - own.n + tok - own.row0, p.lim - 1) : -1;
      }
      const int64_t q_row = p.sq.row0 + tok, q_head = p.head * t.group + gh;
      float c = 0.f;
      const bool warp_live = i * 128 + (warp & 3) * 32 < p.rows;
      if (warp_live) {  // queries, scaled by a power of two
        const uint4* src = reinterpret_cast<const uint4*>(t.q + q_row * t.q_ts + q_head * t.q_hs);
        float big = 0.f;
        if (live) {
#pragma unroll 4
          for (int x = 0; x < D / 8; ++x) {
            const uint4 w = src[x];
            float f[8];
            unpack2<BF16>(w.x, f[0], f[1]), unpack2<BF16>(w.y, f[2], f[3]), unpack2<BF16>(w.z, f[4], f[5]), unpack2<BF16>(w.w, f[6], f[7]);
#pragma unroll
            for (int y = 0; y < 8; ++y) big = fmaxf(big, fabsf(f[y]));
          }
        }
        const int e = row_exponent(big);
        const float down = query_factor(t.scale_log2, e);
        c = score_factor(t.scale_log2, e);
        const uint32_t dst = sm + i * P::kQ + row * 128;
#pragma unroll 1
        for (int x0 = 0; x0 < D / 8; x0 += 4) {
          uint32_t h[16];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint4 w = live ? src[x0 + x] : make_uint4(0, 0, 0, 0);
            float f[8];
            unpack2<BF16>(w.x, f[0], f[1]), unpack2<BF16>(w.y, f[2], f[3]), unpack2<BF16>(w.z, f[4], f[5]), unpack2<BF16>(w.w, f[6], f[7]);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              h[4 * x + y] = BITS == 8 ? pack2<false>(f[2 * y] * down, f[2 * y + 1] * down) : pack2<false>(f[y] * down, f[y + 4] * down);
          }
          if (P::kQTmem) {
            tc_st16(tmem + P::kTmemQ + i * (D / 2) + lanes + x0 * 4, h);
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              sts128(dst + ((x0 + x) >> 3) * (128 * 128) + ((((x0 + x) & 7) ^ (row & 7)) << 4), h[4 * x], h[4 * x + 1], h[4 * x + 2], h[4 * x + 3]);
          }
        }
        if (P::kQTmem) {
          tc_wait_st();
          tc_before();
        } else {
          fence_async_shared();
        }
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar(kQFull + i));
      if (!warp_live) {  // nothing to do but to take part
        for (int j = p.t0; j < p.t1; ++j, ++step) {
          mbar_wait(bar(kSFull + 2 * i + (step & 1)), (step >> 1) & 1, ok);
          if (step > 0) mbar_wait(bar(kODone + i), (step - 1) & 1, ok);
          if (lane == 0) mbar_arrive(bar(kPFull + 2 * i + (step & 1)));
        }
        mbar_wait(bar(kODone + i), (step - 1) & 1, ok);
        finished();
        continue;
      }
      const int see_all = __reduce_min_sync(0xffffffffu, live ? see : INT32_MAX);  // up to here no key is hidden from a row of the warp
      float m = -INFINITY, l = 0.f;
      for (int j = p.t0; j < p.t1; ++j, ++step) {
        const uint32_t pst = step & 1, t_s = tmem + (2 * i + pst) * kKeys + lanes;
        mbar_wait(bar(kSFull + 2 * i + pst), (step >> 1) & 1, ok);
        tc_after();
        uint32_t s[2][32];
        tc_ld32(t_s, s[0]);
        tc_ld32(t_s + 32, s[1]);
        tc_wait_ld();
        const int key0 = j * kKeys;
        if (key0 + kKeys - 1 > see_all) {
#pragma unroll
          for (int x = 0; x < kKeys; ++x)
            if (key0 + x > see) s[x >> 5][x & 31] = 0xFF800000u;
        }
        float top = -INFINITY;
#pragma unroll
        for (int x = 0; x < kKeys; ++x) top = fmaxf(top, __uint_as_float(s[x >> 5][x & 31]));
        top *= c;
        const bool grow = top > m + kGrow || (m == -INFINITY && top > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float r = grow ? ex2(m - top) : 1.f;
          if (grow) m = top;
          l *= r;
          if (j > p.t0) {  // O holds the steps before this one
            mbar_wait(bar(kODone + i), (step - 1) & 1, ok);
            tc_after();
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
              uint32_t o[32];
              tc_ld32(t_o + x, o);
              tc_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * r);
              tc_st32(t_o + x, o);
            }
          }
        }
        const float z = kPShift - (m == -INFINITY ? 0.f : m);
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t ph[16], rest[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const float e0 = ex2(fmaf(__uint_as_float(s[h][x]), c, z));
            const float e1 = ex2(fmaf(__uint_as_float(s[h][x + 1]), c, z));
            l4[(x >> 1) & 3] += e0 + e1;
            ph[x >> 1] = pack2<false>(e0, e1);
            if (P::kRest) rest[x >> 1] = rest_of(ph[x >> 1], e0, e1);
          }
          tc_st16(t_s + h * 16, ph);
          if constexpr (P::kRest) tc_st16(t_s + kKeys / 2 + h * 16, rest);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        // the previous step's product is done by now; seeing each one keeps the barrier's phase known
        if (step > 0) mbar_wait(bar(kODone + i), (step - 1) & 1, ok);
        tc_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + 2 * i + pst));
      }
      mbar_wait(bar(kODone + i), (step - 1) & 1, ok);
      tc_after();
      const int bad = *(volatile int*)bad_of(piece);
      __syncwarp();
      finished();
      if (bad <= see || (p.sq.over && see >= a.max_pages * a.page_size)) l = __uint_as_float(kNaN);
      if (!ok) l = __uint_as_float(kNaN);
      const bool whole = p.t0 == 0 && p.t1 == p.steps, finish = whole && !t.shared;
      const int64_t segment = (int64_t)p.head * W::row_tiles(t, p.sq) + p.rt;  // (with a shared prefix)
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const size_t at = (whole ? (size_t)segment : (size_t)blockIdx.x * 2 + (p.t0 > 0 ? 0 : 1)) * P::kRows + i * 128 + row;
      float* partial = whole ? t.whole : t.partial;
      uint16_t* dst = t.out + q_row * t.o_ts + q_head * t.o_hs;
#pragma unroll 1
      for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        tc_ld32(t_o + x, o);
        tc_wait_ld();
        if (live) {
#pragma unroll
          for (int y = 0; y < 32; y += 8) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[BITS == 8 ? k : (k & 1) * 4 + (k >> 1)] = __uint_as_float(o[y + k]);
            if (finish) {
              *reinterpret_cast<uint4*>(dst + x + y) = make_uint4(pack2<BF16>(f[0] * inv, f[1] * inv), pack2<BF16>(f[2] * inv, f[3] * inv),
                                                                  pack2<BF16>(f[4] * inv, f[5] * inv), pack2<BF16>(f[6] * inv, f[7] * inv));
            } else {
              float4* d4 = reinterpret_cast<float4*>(partial + at * D + x + y);
              d4[0] = make_float4(f[0], f[1], f[2], f[3]);
              d4[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
        __syncwarp();
      }
      if (live) {
        if (!finish)
          (whole ? t.whole_stats : t.stats)[at] = make_float2(m, l);
        else if (t.lse)
          t.lse[q_row * t.nq + q_head] = lse_of(m, l);
      }
      if (tid == 0 && p.t1 == p.steps) {
        if (t.shared)
          t.spans[segment] = Span{whole ? kWhole : p.first_part, (int)blockIdx.x};
        else if (!whole)
          t.ends[blockIdx.x] = SegmentEnd{p.first_part, p.b, p.head, p.rt};
      }
      tc_before();  // O and S have been read before the next piece's products, which wait for its queries or P
    }
  }
  tc_before();
  if (__syncthreads_or(!ok)) {  // (the first wait to run out may be any role's: what it then gives on is taken for good by the others)
    if (tid == 0) kv_flag(a, MOE_KV_TIMEOUT);
    settle();
  }
  tc_after();
  if (warp == kIssueWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(P::kTmemCols));
}

template <int D, int BITS, bool BF16>
moe_status_t launch_tiles_kernel(const KvArgs& kv, const AttArgs& t, cudaStream_t st) {
  using P = TilesPlan<D, BITS, BF16>;
  constexpr auto kernel = attend_tiles_kernel<D, BITS, BF16>;
  const moe_status_t ok = raise_smem<kernel>(P::kSmem);
  if (ok != MOE_OK) return ok;
  // the roles' registers come out of the launch's: with fewer the softmax would wait for its share for good
  static int enough = 0;
  if (!__atomic_load_n(&enough, __ATOMIC_RELAXED)) {
    cudaFuncAttributes at{};
    if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess || at.numRegs < P::kLaunchRegs) return MOE_ERR_CUDA;
    __atomic_store_n(&enough, 1, __ATOMIC_RELAXED);
  }
  kernel<<<t.parts, P::kThreads, P::kSmem, st>>>(kv, t);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int BITS>
moe_status_t launch_tiles(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st) {
  if (dim == 64) return bf16 ? launch_tiles_kernel<64, BITS, true>(kv, t, st) : launch_tiles_kernel<64, BITS, false>(kv, t, st);
  if (dim == 128) return bf16 ? launch_tiles_kernel<128, BITS, true>(kv, t, st) : launch_tiles_kernel<128, BITS, false>(kv, t, st);
  return bf16 ? launch_tiles_kernel<256, BITS, true>(kv, t, st) : launch_tiles_kernel<256, BITS, false>(kv, t, st);
}

}  // namespace
}  // namespace moe
