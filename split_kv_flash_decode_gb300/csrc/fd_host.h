// Argument checks that the host side of the cache calls shares.
#pragma once

#include <cstdint>

#include "../../include/fd.h"

namespace fd {

enum KvKind { kKv16 = 0, kKvE4m3 = 1, kKvE2m1 = 2 };

inline int kv_kind(int dtype) {
  return dtype == FD_F16_E4M3KV                                  ? kKvE4m3
         : dtype == FD_F16_E2M1KV || dtype == FD_BF16_E2M1KV ? kKvE2m1
                                                               : kKv16;
}
inline bool is_bf16(int dtype) { return dtype == FD_BF16 || dtype == FD_BF16_E2M1KV; }
// Bytes of K (or of V) of one token and KV head.
inline int64_t cache_row_bytes(int dtype, int d) {
  const int kind = kv_kind(dtype);
  return kind == kKv16 ? 2 * d : kind == kKvE4m3 ? d : d * 9 / 16;
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A range of bytes.
struct Span {
  uintptr_t at;
  uint64_t n;
};
inline Span span(const void* p, int64_t n) {
  return {reinterpret_cast<uintptr_t>(p), p == nullptr ? 0 : (uint64_t)n};
}
inline bool overlap(const Span& a, const Span& b) {
  return a.n > 0 && b.n > 0 && a.at < b.at + b.n && b.at < a.at + a.n;
}

}  // namespace fd
