// How the gated recurrence shares out a pack: shared by its kernels, its
// workspaces and the CPU tests, which compile it on the host.
#pragma once

#include "wtc_numeric.h"
#include "wtc_tok_internal.h"

namespace wtc {

constexpr int kMostParts = 1024;   // as many maps as a workgroup composes

// Parts of the pack: enough for four waves a vector unit, of 8 tokens at least and kMostParts of them at most; up to 64
// tokens one part, with one launch instead of three and no workspace.  Measured (us forward / backward, bfloat16).
//   One part against parts of 8 tokens, 768 channels, in a captured graph: 24 tokens 7.9 / 12.1 and 11.1 / 12.7, 32 8.7 / 13.7
// and 11.2 / 13.0, 48 10.5 / 16.7 and 11.2 / 12.9, 64 12.2 / 19.8 and 11.2 / 13.0; calls each waited for: 24 20.1 / 24.7 and
// 24.5 / 26.2, 32 20.9 / 26.3 and 24.4 / 26.2, 48 22.7 / 29.2 and 24.3 / 26.2, 64 24.3 / 32.1 and 24.3 / 26.3; one after
// another without waiting as in a graph.  So the forward pass gains up to 56 tokens, at 64 it loses a tenth or nothing; the
// backward pass, which has the same workspace, gains up to 28 (waited for, 32) and from there to 64 loses up to half.  48
// channels: the same.
//   Parts of 64, 32, 16 and 8 tokens at least: 400 x 768 25 / 31, 17.6 / 21, 13.8 / 16, 11.6 / 13.3; 12544 x 384 30 / 42, 25 /
// 35, 23.4 / 31.3, 23.4 / 31.2 (784 parts are enough there).  For two waves a unit and for four: 130219 x 384 107 / 164 and
// 99.7 / 154, 2 x 65536 x 512 147 / 219 and 149 / 216, 12544 x 1024 36.3 / 49.5 and 37.1 / 47.8; for eight the two large ones do
// not change.
//   Long packs of few channels are held back by kMostParts: 512 C threads, each with T / 1024 tokens one after another, twice.
// 100000 tokens of 16, 48 and 96 channels 36.5 / 45, 37 / 51 and 38.5 / 52, where a copy of their bytes takes 1.9 / 3.1, 5.7 /
// 9.4 and 11 / 19; 1000000 of 16, 48, 96 and 192 242 / 362, 237 / 463, 273 / 513 and 430 / 669, for 19 / 31, 57 / 94, 113 /
// 189 and 227 / 378.
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
