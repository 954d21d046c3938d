"""Host arithmetic of the layer norm, gated scan and experts operators, compiled from the
headers that the kernels include, with UndefinedBehaviorSanitizer."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "memory_bound_cnn_amd", "csrc")


def run(tmp_path, program):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(program)
    subprocess.run([cxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", f"-I{CSRC}",
                    f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return r.stdout


def test_gated_scan_parts_cover_every_pack(tmp_path):
    """Parts follow one another from token 0 to T - 1 with int arithmetic that does not overflow, up to the largest pack."""
    out = run(tmp_path, r"""
#include <cstdio>
#include "wtc_tok_scan.h"

static long check(long long T, int C) {
    const wtc::ScanSplit s = wtc::scan_split(T, C);
    if (s.parts < 1 || s.parts > wtc::kMostParts || s.len % wtc::kScanKept != 0) return 1;
    int next = 0;
    for (int part = 0; part < s.parts; ++part) {
        const int first = part * s.len, end = wtc::part_end(first, s.len, (int)T);
        if (first != next || end > T || (T > 0 && end <= first)) return 1;
        next = end;
    }
    return next == T ? 0 : 1;
}

int main() {
    const int channels[] = {1, 2, 3, 16, 48, 96, 384, 387, 512, 2048, 262143, 262144, 1 << 20};
    const long long limit = (1LL << 31) - (1 << 10);   // sizes from here on are refused
    long bad = 0, n = 0;
    for (int C : channels) {
        for (long long T = 0; T < 3000; ++T, ++n) bad += check(T, C);
        for (long long T = limit - 9400; T < limit; ++T, ++n) bad += check(T, C);
        for (int b = 12; b < 31; ++b)
            for (int i = -9; i <= 9; ++i, ++n) bad += check((1LL << b) + i, C);
    }
    printf("%ld of %ld bad\n", bad, n);
    return bad != 0;
}
""")
    assert out.startswith("0 of ")


def test_tiles_of_rows_stay_inside_of_them(tmp_path):
    """Each row of a segment is in one tile, and no tile, of whatever number, reaches past its end, up to the most rows."""
    out = run(tmp_path, r"""
#include <climits>
#include <cstdio>
#include "wtc_tok_segment.h"

template <int SIZE>
static long check(int b, int e) {
    long bad = 0;
    const int tiles = e > b ? (int)(((long long)e - b + SIZE - 1) / SIZE) : 0;
    const int near[] = {-1, 0, 1, 2, tiles - 2, tiles - 1, tiles, tiles + 1, tiles + 512, INT_MAX / SIZE - 1, INT_MAX / SIZE + 1,
                        INT_MAX / SIZE + 514, INT_MAX / 2, INT_MAX};
    for (int t : near) {
        const wtc::product::Rows r = wtc::product::rows_of<SIZE>(7, b, e, t);
        const long long from = (long long)b + (long long)t * SIZE, to = from + SIZE < e ? from + SIZE : e;
        const int want = t >= 0 && from < to ? (int)(to - from) : 0;
        bad += r.expert != 7 || r.count != want || (want && r.start != from);
    }
    return bad;
}

int main() {
    const int most = INT_MAX - (1 << 16);   // as many rows as a call may have
    const int at[] = {0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 1000, 1 << 20, (1 << 30) - 1, 1 << 30,
                      most - 513 * 256, most - 257, most - 256, most - 1, most};
    long bad = 0, n = 0;
    for (int b : at)
        for (int e : at) bad += check<16>(b, e) + check<32>(b, e) + check<64>(b, e) + check<128>(b, e) + check<256>(b, e), ++n;
    printf("%ld of %ld bad\n", bad, n);
    return bad != 0;
}
""")
    assert out.startswith("0 of ")
