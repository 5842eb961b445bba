"""The order in which the split and rows kernels visit a tile's rows (``csrc/exact_order.cuh``, compiled
here by the host compiler): every warp's step has between 1 and all of its rows behind it, in one piece,
and the steps of a team together have every row that a token sees, once."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "rank_kv_cache_isvd_b200", "csrc")

WALK = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "exact_order.cuh"
using namespace iskv;

static long long walked = 0;

static void fail(const char *what, int n, int ql, int i0, int tpt, int window, int sinks, int wr, int team, int c) {
    std::printf("%s: n %d ql %d i0 %d tpt %d window %d sinks %d wr %d team %d place %d\n", what, n, ql, i0, tpt,
                window, sinks, wr, team, c);
    std::exit(1);
}

static void item(int n, int ql, int i0, int tpt, int window, int sinks, int wr, int team) {
    const int i1 = i0 + tpt < ql ? i0 + tpt : ql, rs = wr * team;
    const ExactOrder o = ex_order(n, ql, i0, i1, window, sinks, wr);
    if (o.C > ex_most_rows(window, sinks, tpt, n, wr)) fail("longer than reckoned", n, ql, i0, tpt, window, sinks, wr, team, o.C);
    std::vector<int> times(n + 1, 0);
    const int steps = (o.C + rs - 1) / rs;
    for (int st = 0; st < steps; ++st)
        for (int tw = 0; tw < team; ++tw) {
            const int c = st * rs + tw * wr;
            if (c >= o.C) continue;
            ++walked;
            const int seen = ex_seen(o, c, wr);
            if (seen < 1 || seen > wr) fail("rows of a step", n, ql, i0, tpt, window, sinks, wr, team, c);
            if (c < o.skp && c + wr > o.skp) fail("a step of both parts", n, ql, i0, tpt, window, sinks, wr, team, c);
            for (int r = 0; r < seen; ++r) {
                const int j = ex_row(o, c) + r;
                if (j < 0 || j >= n) fail("row out of range", n, ql, i0, tpt, window, sinks, wr, team, c);
                ++times[j];
            }
        }
    for (int j = 0; j < n; ++j) {
        bool visible = false;
        for (int i = i0; i < i1; ++i) {
            const int p = n - ql + i;
            visible |= j <= p && (j < sinks || j > p - window);
        }
        if (times[j] != (visible ? 1 : 0)) fail("visits of a row", n, ql, i0, tpt, window, sinks, wr, team, j);
    }
}

int main() {
    const int windows[] = {1, 5, 16, 33, 100, 300, 1 << 24};
    const int lengths[] = {0, 1, 2, 15, 16, 17, 31, 47, 64, 100, 130, 200, 331, 517};
    const int tokens[] = {1, 2, 3, 8, 40};
    std::vector<int> sinks;
    for (int s = 0; s <= 70; ++s) sinks.push_back(s);
    sinks.push_back(130);
    for (int wr : {ex_warp_rows(true), ex_warp_rows(false)})
        for (int team = 1; team <= 8; team *= 2)
            for (int window : windows)
                for (int n : lengths)
                    for (int ql : tokens)
                        for (int s : sinks)
                            for (int tpt : {1, 2, 8, 64})
                                for (int i0 = 0; i0 < ql; i0 += tpt)
                                    item(n, ql, i0, tpt, window, s < n ? s : n, wr, team);
    std::printf("%lld steps\n", walked);
    return walked > 1000000 ? 0 : 2;
}
"""


def test_steps_have_rows_and_cover_what_is_seen(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(WALK)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout


def test_wait_limits_are_checked():
    import rank_kv_cache_isvd_b200 as iskv
    assert iskv.iskv_exact_wait_limit(-1) == iskv.ISKV_ERR_INVALID_ARG
    assert iskv.iskv_exact_wait_limit(1) == 0 and iskv.iskv_exact_wait_limit() == 0
