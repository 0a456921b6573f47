// What the kernels over 8-bit rows share: the types of a call, checks of rows with a pitch,
// and the groups of elements that they move. A row t of a checkpoint stands for s_t q_t, q
// whole numbers of [-127, 127], s_t a power of two; s_t = 0 marks a row that takes no part,
// s_t = NaN one that held an infinity or a NaN.
#pragma once
#include <algorithm>

#include "row_ops.hpp"

namespace kfac {

typedef unsigned short v4us __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v8f __attribute__((ext_vector_type(8)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef v4s __attribute__((address_space(3))) lds_v4s;

inline int dtype_bytes(kfac_dtype d) { return d == KFAC_F32 ? 4 : 2; }
inline bool row_dtype(kfac_dtype d) { return d == KFAC_F16 || d == KFAC_BF16 || d == KFAC_F32; }

// Rows of `width` elements of `size` bytes, `ld` elements apart.
struct RowsOf {
  const void* at;
  int64_t rows, width, ld;
  int size;
  const char* name;
  bool empty() const { return rows <= 0 || width <= 0; }
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(at); }
  uintptr_t end() const { return begin() + (uintptr_t(rows - 1) * ld + width) * size; }
};

inline kfac_status check_rows(const RowsOf& r) {
  if (r.empty()) return KFAC_OK;
  if (!r.at) return fail(KFAC_ERR_INVALID, "%s is NULL", r.name);
  if (r.begin() % r.size) return fail(KFAC_ERR_INVALID, "%s is misaligned", r.name);
  if (r.rows > 1 && r.ld < r.width) return fail(KFAC_ERR_INVALID, "the rows of %s overlap", r.name);
  return KFAC_OK;
}

// Whether two sets of rows share a byte. Sets whose ranges cross but whose rows lie between each
// other's (parts of wider rows at the same pitch) do not.
inline bool rows_share(const RowsOf& a, const RowsOf& b) {
  if (a.empty() || b.empty() || !a.at || !b.at || a.end() <= b.begin() || b.end() <= a.begin()) return false;
  const int64_t pitch = a.ld * a.size;
  if (a.rows == 1 || b.rows == 1 || pitch != b.ld * b.size) return true;
  const int64_t wa = a.width * a.size, wb = b.width * b.size;
  int64_t off = static_cast<int64_t>(b.begin() - a.begin()) % pitch;
  if (off < 0) off += pitch;
  return off < wa || off + wb > pitch;
}

// Waits until at most N of this wave's loads are on their way and its LDS operations are done, then for the
// other waves.
template <int N>
__device__ inline void arrive() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The part of a workspace that a call uses, as one row.
inline RowsOf scratch(void* ws, size_t need) { return {ws, need ? 1 : 0, static_cast<int64_t>(need), 0, 1, "workspace"}; }

// Refuses a call two of whose buffers share bytes, if one of them is written: outputs first, `written` of them.
inline kfac_status check_apart(const RowsOf* const* buf, int n, int written) {
  for (int a = 0; a < written; ++a)
    for (int b = a + 1; b < n; ++b)
      if (rows_share(*buf[a], *buf[b])) return fail(KFAC_ERR_INVALID, "%s and %s overlap", buf[a]->name, buf[b]->name);
  return KFAC_OK;
}
template <size_t N>
kfac_status check_apart(const RowsOf* const (&buf)[N], int written) {
  return check_apart(buf, static_cast<int>(N), written);
}

// A launch has fewer than 2^32 threads: most blocks of 256, in whole eights.
constexpr int64_t kMostBlocks = (int64_t(1) << 24) - 8;

// The element types as the kernels take them.
template <class F>
kfac_status with_row_type(kfac_dtype d, F f) {
  if (d == KFAC_F32) return f(float{});
  if (d == KFAC_BF16) return f(__bf16{});
  return f(_Float16{});
}

}  // namespace kfac
