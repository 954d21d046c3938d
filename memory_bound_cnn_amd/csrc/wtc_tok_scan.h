// How the gated recurrence shares out a pack: shared by its kernels, its
// workspaces and the CPU tests, which compile it on the host.
#pragma once

#include "wtc_numeric.h"
#include "wtc_tok_internal.h"

namespace wtc {

constexpr int kMostParts = 1024;   // as many maps as a workgroup composes

// Parts of the pack: enough for four waves a vector unit, of 8 tokens at least; one where that is sooner done than three
// kernels.  Measured (us forward / backward, bfloat16): 768 channels, one part against parts of 8 tokens, 24 tokens 7.9 /
// 11.5 and 11.2 / 13.2, 32 8.8 / 13.0 and 11.6 / 13.2, 64 12.5 / 18.8 and 11.6 / 13.4 (one launch instead of three is the
// host's gain), 100 16.4 / 25 and 11.6 / 13.3, 400 52 / 80 and 11.6 / 13.3.  Parts of 64, 32, 16 and 8 tokens at least: 400 x
// 768 25 / 31, 17.6 / 21, 13.8 / 16, 11.6 / 13.3; 12544 x 384 30 / 42, 25 / 35, 23.4 / 31.3, 23.4 / 31.2 (784 parts are enough
// there).  For two waves a unit and for four: 130219 x 384 107 / 164 and 99.7 / 154, 2 x 65536 x 512 147 / 219 and 149 / 216,
// 12544 x 1024 36.3 / 49.5 and 37.1 / 47.8; for eight the two large ones do not change (kMostParts).
struct ScanSplit {
    int parts, len;   // parts begin at the multiples of len
};
inline ScanSplit scan_split(long long T, int C) {
    const long long pairs = (C + 1) / 2, want = (262144 + pairs - 1) / pairs, most = T <= 64 ? 1 : (T + 7) / 8;
    long long parts = want < most ? want : most;
    parts = parts < 1 ? 1 : parts > kMostParts ? kMostParts : parts;
    ScanSplit s;
    s.len = (int)(((T + parts - 1) / parts + kScanKept - 1) / kScanKept * kScanKept);
    s.parts = s.len < 1 ? 1 : (int)((T + s.len - 1) / s.len);
    return s;
}
// The end of the part that begins at `first`: first + len may be beyond 2^31, by up to kMostParts kScanKept.
WTC_HD int part_end(int first, int len, int T) { return first + (T - first < len ? T - first : len); }

}  // namespace wtc
