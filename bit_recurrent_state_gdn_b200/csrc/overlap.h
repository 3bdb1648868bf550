// Whether the arrays of a call share memory, on the host.
#pragma once

#include <algorithm>
#include <cstdint>

#include "layer_args.h"
#include "status.h"

namespace gdnq {

// The arrays of one call, and the check that no output meets another array. Decided exactly where one
// of the two fills its range without gaps or both have the same strides (slices of one buffer);
// otherwise, two arrays with gaps and different strides, they are taken to be apart.
class Arrays {
 public:
  void tokens(const gdn_tokens* t, const char* name, int64_t B, int64_t L, int64_t H, int64_t D,
              unsigned elem, bool output) {
    if (!t || !t->ptr || B * H == 0 || L == 0) return;
    Array& a = list[n++];
    a.name = name;
    a.p = reinterpret_cast<uintptr_t>(t->ptr);
    a.run = a.span = D * elem;
    a.output = output;
    const int64_t strides[3] = {t->sb, t->sl, t->sh}, sizes[3] = {B, L, H};
    for (int i = 0; i < 3; ++i) {
      const bool moves = sizes[i] > 1 && strides[i] > 0;
      a.dims[i] = {moves ? strides[i] * (int64_t)elem : 0, moves ? sizes[i] : 1};
    }
    std::sort(a.dims, a.dims + 3, [](const Dim& p, const Dim& q) { return p.stride > q.stride; });
    a.solid = true;  // every dimension steps from one end of what the smaller ones fill to the next
    for (int i = 2; i >= 0; --i) {
      a.solid = a.solid && (a.dims[i].size == 1 || a.dims[i].stride == a.span);
      a.span += a.dims[i].stride * (a.dims[i].size - 1);
    }
  }
  void dense(const void* p, const char* name, size_t bytes, bool output) {
    if (!p || !bytes) return;
    list[n++] = Array{name, reinterpret_cast<uintptr_t>(p), (int64_t)bytes, (int64_t)bytes,
                      {{0, 1}, {0, 1}, {0, 1}}, output, true};
  }
  // `out` may be `in`; what else they share is refused.
  gdn_status check(const void* out = nullptr, const void* in = nullptr) const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j) {
        const Array &a = list[i], &b = list[j];
        if (!a.output && !b.output) continue;
        if (out && out == in && a.p == b.p && a.p == reinterpret_cast<uintptr_t>(out)) continue;
        if (meet(a, b))
          return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", a.output ? a.name : b.name,
                      a.output ? b.name : a.name);
      }
    return GDN_OK;
  }

 private:
  struct Dim {
    int64_t stride, size;  // bytes, indexes
  };
  struct Array {
    const char* name;
    uintptr_t p;
    int64_t run, span;  // bytes that follow one another, bytes from the first to behind the last
    Dim dims[3];        // the largest stride first
    bool output, solid;
  };
  Array list[16];
  int n = 0;

  static bool meet(const Array& a, const Array& b) {
    const int64_t d = (int64_t)(b.p - a.p);
    if (d >= a.span || -d >= b.span) return false;
    if (b.solid) return touches(a, 0, d, d + b.span);
    if (a.solid) return touches(b, 0, -d, -d + a.span);
    for (int i = 0; i < 3; ++i)
      if (a.dims[i].stride != b.dims[i].stride || a.dims[i].size != b.dims[i].size) return false;
    return a.run == b.run && meets_shifted(a, 0, d);
  }

  // Whether dimensions k and later of a, from offset 0 on, have a byte in [lo, hi).
  static bool touches(const Array& a, int k, int64_t lo, int64_t hi) {
    if (hi <= 0) return false;
    while (k < 3 && a.dims[k].size == 1) ++k;
    if (k == 3) return lo < a.run;
    const int64_t s = a.dims[k].stride, last = a.dims[k].size - 1;
    int64_t inner = a.run;  // bytes that the later dimensions span
    for (int i = k + 1; i < 3; ++i) inner += a.dims[i].stride * (a.dims[i].size - 1);
    // index i begins at i s: one that begins in the range has a byte there; of those before it, the
    // nearest ones may reach in (one, or a few of an input whose rows share memory)
    const int64_t from = lo <= 0 ? 0 : (lo + s - 1) / s;
    if (from <= last && from * s < hi) return true;
    for (int64_t i = std::min(from - 1, last), tries = 0; i >= 0 && i * s + inner > lo && tries < 8; --i, ++tries)
      if (touches(a, k + 1, lo - i * s, hi - i * s)) return true;
    return false;
  }

  // Whether a meets itself moved by d bytes.
  static bool meets_shifted(const Array& a, int k, int64_t d) {
    while (k < 3 && a.dims[k].size == 1) ++k;
    if (k == 3) return d < a.run && -d < a.run;
    const int64_t s = a.dims[k].stride, size = a.dims[k].size;
    const int64_t i = d / s;  // indexes differ by this, or by one more or less
    for (int64_t j = i - 1; j <= i + 1; ++j)
      if (j > -size && j < size && meets_shifted(a, k + 1, d - j * s)) return true;
    return false;
  }
};

}  // namespace gdnq
