// Host-side pieces of the 8-bit key-value cache operators: the arguments as the kernels take them,
// and their checks.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/w8a8.h"

namespace w8a8 {

struct Kv8Step {
  const int* row0;
  const int* kv_len;
  const int* page_table;
  int seqs, tokens, max_tokens, table_width;
};

inline Kv8Step kv8_step_of(const kv8_step_t& s) {
  return Kv8Step{s.row0, s.kv_len, s.page_table, s.seqs, s.tokens, s.max_tokens, s.table_width};
}

inline bool kv8_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of 16-bit heads: a 16-byte aligned pointer and a stride (in elements) of whole 16-byte
// vectors that holds the row.
inline int kv8_check_rows(const void* p, long long stride, int heads, int head_dim) {
  if (!p || stride < (long long)heads * head_dim || stride > (1ll << 31)) return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(p, 16) || stride % 8 != 0) return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

int kv8_check_dims(int kv_heads, int head_dim);
int kv8_check_cache(const kv8_cache_t* c);
int kv8_check_step(const kv8_step_t* s, const kv8_cache_t* c);
// Workspace: non-null, aligned, at least the status header.
int kv8_check_ws(const void* ws, size_t ws_bytes, size_t need);
// prep may be NULL (no norm, no rotation).
int kv8_check_prep(const qk_prep_t* p, int head_dim);

// Most pages that a sequence of max_tokens rows can touch: its rows may begin at the end of one.
inline int kv8_pages_of(int max_tokens, int page_tokens) { return (max_tokens + page_tokens - 2) / page_tokens + 1; }

}  // namespace w8a8
