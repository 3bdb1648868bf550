// Gated scan: when sequences are split into spans.
#include <algorithm>

#include "scan_kernels.cuh"

namespace gdnq {

// Units (64 channels of a sequence) too few for clusters of eight CTAs to fill the machine, and long:
// spans of at least 128 tokens, as many as two CTAs per SM take at once. Against one cluster a unit,
// bf16, forward / backward: 64 channels x 131072 tokens 33 / 39 us (292 / 579), 232 x 78755 62 / 81
// (211 / 415), 256 x 32768 31 / 37 (78 / 163), 1024 x 32768 92 / 125 (107 / 206), 1152 x 60000 (18
// units) 168 / 241 (199 / 378); 19 units of 32768 tokens take 113 / 209 in clusters.
// GDN_SCAN_SPLIT, where two launches begin to pay: 256 channels x 2048 tokens 13.1 / 16.4 us in spans
// (9.0 / 14.6), x 3136 13.5 / 16.6 (14.6 / 20.8), x 4096 13.6 / 16.6 (14.5 / 22.9), x 6000 16.9 / 16.7
// (18.7 / 31.1); 1024 channels x 3136 20.8 / 22.9 (18.7 / 26.1), x 4096 21.2 / 22.9 (18.7 / 29.1).
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
