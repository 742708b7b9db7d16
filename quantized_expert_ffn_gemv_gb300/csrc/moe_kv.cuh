// Pieces shared by the kernels of the quantised paged cache: the pool's
// layout, the batch's arrays, and the checks of their contents.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "moe_model.h"

namespace moe {

constexpr int kKvTile = 32;  // tokens of a tile

__host__ __device__ constexpr int kv_row_bytes(int dim, int bits) { return dim * bits / 8; }
// K (or V) half of a tile: 32 value rows and their scales.
__host__ __device__ constexpr int kv_half_bytes(int dim, int bits) { return kKvTile * kv_row_bytes(dim, bits) + 2 * dim; }
__host__ __device__ constexpr int kv_tile_bytes(int dim, int bits) { return 2 * kv_half_bytes(dim, bits); }

// Where chunk c of value row r lies: c ^ (kv_turn(r) & (chunks - 1)).  Its
// three bits are such that the rows a quarter-warp reads together (8
// consecutive ones for K fragments, every other one for V fragments) fall on
// different 16-byte bank groups.
__host__ __device__ constexpr int kv_turn(int r) { return (((r >> 2) ^ r) & 1) << 2 | (r & 2) | ((r >> 2) & 1); }

// What a kernel needs of a cache and a batch, by value.
struct KvArgs {
  uint8_t* data;
  int32_t* status;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int n_pages, page_size, page_shift;  // page_shift: log2(page_size) or -1
  int heads, table_stride, max_pages, n_seqs, n_tokens, max_tokens;
  size_t page_bytes, head_bytes;
};

__device__ __forceinline__ void kv_flag(const KvArgs& a, int bit) { atomicOr(a.status, bit); }

__device__ __forceinline__ int kv_page_of(const KvArgs& a, int pos) {
  return a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
}

// The sequence whose new tokens hold row t, or -1 (a row behind the last
// sequence, or arrays that do not ascend).  A batch of one token a sequence
// answers after one probe.
__device__ __forceinline__ int kv_seq_of(const KvArgs& a, int t) {
  int lo = 0, hi = a.n_seqs - 1;
  const int guess = t < hi ? t : hi;
  const int c0 = __ldg(a.cu + guess), c1 = __ldg(a.cu + guess + 1);
  if (c0 <= t && t < c1) return guess;
  if (t < c0)
    hi = guess - 1;
  else
    lo = guess + 1;
  while (lo <= hi) {
    const int mid = (lo + hi) >> 1;
    if (t < __ldg(a.cu + mid))
      hi = mid - 1;
    else if (t >= __ldg(a.cu + mid + 1))
      lo = mid + 1;
    else
      return mid;
  }
  return -1;
}

// Whether a sequence's new tokens c0 .. c1 - 1 can be: an ascending share of the rows, no more of them than the call or the sequence has.
__device__ __forceinline__ bool kv_seq_ok(const KvArgs& a, int c0, int c1, int len) {
  return c0 >= 0 && c1 >= c0 && c1 <= a.n_tokens && c1 - c0 <= min(a.max_tokens, len);
}
__device__ __forceinline__ bool kv_seq_ok(const KvArgs& a, int b) {
  return kv_seq_ok(a, __ldg(a.cu + b), __ldg(a.cu + b + 1), __ldg(a.lens + b));
}

// The 32-token tile that holds position pos (>= 0) of sequence b, head 0, or
// NULL for a bad page.
__device__ __forceinline__ uint8_t* kv_tile_of(const KvArgs& a, int b, int pos, int tile_bytes) {
  const int pi = kv_page_of(a, pos);
  if (pi >= a.max_pages) return nullptr;
  const int page = __ldg(a.table + (size_t)b * a.table_stride + pi);
  if ((unsigned)page >= (unsigned)a.n_pages) return nullptr;
  return a.data + (size_t)page * a.page_bytes + (size_t)((pos - pi * a.page_size) / kKvTile) * tile_bytes;
}

// Host: checks of a cache and a batch, and their kernel form; rows of heads; the SM count (looked up once a device).
moe_status_t kv_args(const moe_kv_cache_t* c, const moe_kv_batch_t* b, KvArgs* out);
bool heads_ok(const moe_heads_t* h, int dim);
bool out_heads_ok(const moe_heads_t* h, int n_heads, int n_tokens, int dim);
constexpr int kMaxDevices = 64;
moe_status_t device_sms(int* sms);
// Raises the shared memory that a kernel may use on the current device, once a
// device; always to the same size, so that calls at the same time agree.
template <auto KERNEL>
moe_status_t raise_smem(int bytes) {
  static int raised[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
  if (__atomic_load_n(&raised[dev], __ATOMIC_RELAXED) >= bytes) return MOE_OK;
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return MOE_ERR_CUDA;
  __atomic_store_n(&raised[dev], bytes, __ATOMIC_RELAXED);
  return MOE_OK;
}

template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
  if (BF16) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = f.x;
    b = f.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace moe
