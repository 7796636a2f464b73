"""How head norms split a token's heads over groups of lanes (csrc/head_split.h),
walked on the host: every head once, no part that begins behind the last head, as the
kernel's walk over a part ends only by counting its heads down."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "moe_routing_capacity_gb300", "csrc", "head_split.h")

WALK = r"""
#include <cstdio>
#include <initializer_list>
#include "%s"
using namespace moe;

static bool covers(int n, int parts) {      // the forward's runs of neighbours
    const HeadRuns r = head_runs(n, parts);
    if (n == 0) return r.runs == 0;
    if (r.runs < 1 || r.runs > parts || r.each < 1) return false;
    int next = 0;
    for (int i = 0; i < r.runs; ++i) {
        const int h = i * r.each, left = n - h < r.each ? n - h : r.each;
        if (h != next || left <= 0) return false;
        next = h + left;
    }
    return next == n;
}

// The gradient's parts: heads i, i + parts, ...
static bool parts_ok(int n, int parts) { return n == 0 ? parts == 0 : parts >= 1 && parts <= n; }

int main() {
    for (int n = 1; n <= 4096; ++n)
        for (int parts = 1; parts <= n; ++parts)
            if (!covers(n, parts)) return std::printf("%%d heads in %%d parts\n", n, parts), 1;
    const int64_t tokens[] = {1, 2, 3, 7, 16, 33, 70, 129, 257, 600, 1023, 1400, 1457, 2000, 2048, 2707, 2780, 2900,
                              2993, 3000, 3157, 3892, 4096, 4323, 6000, 8192, 12001, 16384, 30011, 65536, 262144,
                              1 << 20, 1ll << 31, 1ll << 40};
    long walks = 0;
    for (int sms : {148, 152})
        for (int lanes = 4; lanes <= 32; lanes *= 2)
            for (int64_t T : tokens)
                for (int n = 1; n <= 65536; n += n < 1024 ? 1 : n %% 61 + 1)
                    for (int other : {0, 1, 8, n}) {
                        for (int keys = 0; keys < 2; ++keys) {
                            const int hq = keys && other ? other : n, hk = keys && other ? n : other;
                            const HeadParts p = head_parts(T, hq, hk, lanes, (int64_t)sms * 512);
                            if (!parts_ok(hq, p.q) || !parts_ok(hk, p.k) || !covers(hq, p.q) || !covers(hk, p.k))
                                return std::printf("%%lld tokens, %%d + %%d heads, %%d lanes, %%d SMs\n", (long long)T,
                                                   hq, hk, lanes, sms), 1;
                            ++walks;
                        }
                    }
    std::printf("%%ld\n", walks);
    return 0;
}
"""


def test_every_head_is_in_one_part(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    (tmp_path / "w.cpp").write_text(WALK % HEADER)
    subprocess.run([cxx, "-O2", "-std=c++17", str(tmp_path / "w.cpp"), "-o", str(tmp_path / "w")], check=True)
    r = subprocess.run([str(tmp_path / "w")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 1000000
