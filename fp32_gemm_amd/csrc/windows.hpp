// windows.hpp -- the bytes that an operand covers, and whether two share any.
#pragma once

#include <cstdint>

namespace fp32gemm {

// Bytes of a rows x cols window, from its first element to its last.
inline long long extent(long long rows, long long cols, long long ld, int es) {
  return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * es : 0;
}
inline bool overlap(const void* a, long long an, const void* b, long long bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an > 0 && bn > 0 && x < y + static_cast<uintptr_t>(bn) && y < x + static_cast<uintptr_t>(an);
}

struct Window {
  const void* at;
  long long bytes;
};
inline bool meet(const Window& a, const Window& b) { return overlap(a.at, a.bytes, b.at, b.bytes); }

}  // namespace fp32gemm
