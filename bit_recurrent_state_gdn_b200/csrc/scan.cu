// Gated scan: when sequences are split into spans.
#include <algorithm>

#include "scan_kernels.cuh"

namespace gdnq {

// Units (64 channels of a sequence) too few for clusters of eight CTAs to fill the machine, and long:
// spans of at least 128 tokens, as many as two CTAs per SM take at once. Against one cluster a unit:
// 232 channels x 78755 tokens 57 us / 183, 256 channels x 32768 backward 42 / 167, 1024 x 32768
// backward 128 / 207, 1024 x 60000 147 / 168; at 1152 channels (18 units) 162 / 168.
size_t scan_spans(ScanArgs& a) {
  a.span_tokens = 0;
  a.spans_per_unit = 0;
  const int64_t units = (int64_t)a.B * ((a.C + kScanSlab - 1) / kScanSlab);
  if (units < 1 || units * 8 >= kSms || a.L < GDN_SCAN_SPLIT) return 0;
  constexpr int kGrain = 128;  // whole tiles of every kernel, and kept chunks
  const int64_t want = (2 * kSms) / units, tokens = (a.L + want - 1) / want;
  a.span_tokens = (int)((tokens + kGrain - 1) / kGrain * kGrain);
  a.spans_per_unit = (a.L + a.span_tokens - 1) / a.span_tokens;
  return (size_t)units * (size_t)(a.spans_per_unit + 1) * 32 * (sizeof(SpanLink) + sizeof(SpanDecay));
}

}  // namespace gdnq
