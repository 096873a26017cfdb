// Host-side argument checks shared by the C-ABI calls of qat_mx.h and qat_kv.h.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/qat.h"

#define QAT_API extern "C" __attribute__((visibility("default")))

#define QAT_CHECK(x)               \
  do {                             \
    int32_t _st = (x);             \
    if (_st != QAT_OK) return _st; \
  } while (0)

namespace qat {

// Kernels address each matrix operand with 32-bit byte offsets.
constexpr int64_t kMaxOperandBytes = 0x7FFFFFF0;
constexpr int64_t kMaxCount = int64_t(1) << 30;

// A written or read region of device memory; n == 0 or p == nullptr: none.
struct Span {
  const void* p;
  size_t n;
};

inline bool spans_meet(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// No written region meets a read one or another written one.
inline int32_t check_spans(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* v = w + 1; v != written.end(); ++v)
      if (spans_meet(*w, *v)) return QAT_ERR_ALIAS;
    for (const Span& r : read)
      if (spans_meet(*w, r)) return QAT_ERR_ALIAS;
  }
  return QAT_OK;
}

inline int32_t check_required(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return QAT_ERR_NULL;
  return QAT_OK;
}

inline int32_t check_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 15) return QAT_ERR_ALIGN;
  return QAT_OK;
}

// Bytes from the first element to the end of the last row of `rows` rows of
// `cols` elements, `ld` elements apart.
inline size_t strided_bytes(int64_t rows, int64_t ld, int64_t cols, int64_t elem) {
  return rows > 0 ? (size_t)(((rows - 1) * ld + cols) * elem) : 0;
}

// The rows of two strided operands (`ra`, `rb` elements of 2 bytes, `lda`, `ldb`
// apart) are apart: their spans do not meet, or both have one stride and the
// rows lie side by side in it (slices of one packed projection).
inline int32_t check_rows_apart(const Span& a, int64_t lda, int64_t ra, const Span& b, int64_t ldb, int64_t rb) {
  if (!spans_meet(a, b)) return QAT_OK;
  if (lda != ldb) return QAT_ERR_ALIAS;
  const int64_t stride = lda * 2;
  int64_t off = ((int64_t)((uintptr_t)b.p - (uintptr_t)a.p)) % stride;   // of b's rows behind a's
  if (off < 0) off += stride;
  return off >= ra * 2 && off + rb * 2 <= stride ? QAT_OK : QAT_ERR_ALIAS;
}

}  // namespace qat
