// Reading a batch's device arrays (fp8_kv_batch_t) inside kernels, kept within
// the buffers whatever the arrays hold.
#pragma once

#include "fp8lin_block.h"
#include "internal.h"

namespace fp8lin {
namespace {

struct KVSeq {
  int first;  // row of its first new token
  int n;      // new tokens
  int start;  // position of the first new one
  int len;    // tokens in the cache (0 <= start, start + n = len)
};

__device__ __forceinline__ KVSeq kv_seq(const fp8_kv_batch_t& b, int block_size, int i) {
  KVSeq s;
  s.first = max(0, min(b.cu_tokens[i], b.tokens));
  const int end = max(s.first, min(b.cu_tokens[i + 1], b.tokens));
  s.len = max(0, min(b.lens[i], b.max_len));
  s.n = min(min(end - s.first, b.max_new), s.len);
  s.start = s.len - s.n;
  return s;
}

// The same for an i that is the same in every lane: scalar values.
__device__ __forceinline__ KVSeq kv_seq_uniform(const fp8_kv_batch_t& b, int block_size, int i) {
  const KVSeq s = kv_seq(b, block_size, i);
  return {__builtin_amdgcn_readfirstlane(s.first), __builtin_amdgcn_readfirstlane(s.n),
          __builtin_amdgcn_readfirstlane(s.start), __builtin_amdgcn_readfirstlane(s.len)};
}

// Block of sequence i that holds its tokens [block_at * block_size, ...), or
// -1.  block_at < table_width (max_len <= table_width * block_size).
__device__ __forceinline__ int kv_block(const fp8_kv_cache_t& c, const fp8_kv_batch_t& b, int i, int block_at) {
  const int block = b.block_table[(int64_t)i * b.table_width + block_at];
  return (uint32_t)block < (uint32_t)c.num_blocks ? block : -1;
}

}  // namespace
}  // namespace fp8lin
