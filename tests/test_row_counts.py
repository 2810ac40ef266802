"""Counts of receive rows near the largest int: the cut of an expert's rows into tiles on the CPU, from the kernels'
own header, and the refusal of what 32 bits cannot count."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "moe_experts.cuh"

int main() {
    long long bad = 0, seen = 0;
    const int wide[] = {64, 128, 256, 320, 384}, units[] = {16, 32, 64};
    auto check = [&](int rows, int columns, int unit) {
        const long long r = rows;
        const int tiles = moe::tiles_of(rows, columns);
        if (tiles != (r + columns - 1) / columns) { ++bad; return; }
        const long long per = moe::rows_of_tile(rows, tiles, unit);
        ++seen;
        // every tile has a row, none more than a tile holds, together they have them all
        if (per < 1 || per > columns || per % unit != 0 || per * (tiles - 1) >= r || per * tiles < r) ++bad;
    };
    for (int columns : wide)
        for (int unit : units) {
            for (int i = 0; i < 3000; ++i) check(MOE_MAX_EXPERT_ROWS - i, columns, unit);
            for (int i = 1; i < 3000; ++i) check(i, columns, unit);
            for (long long r = 1; r <= MOE_MAX_EXPERT_ROWS; r = r * 5 / 4 + 1) check((int)r, columns, unit);
        }
    for (int i = 0; i < 3000; ++i)
        if (moe::blocks_of_128(MOE_MAX_EXPERT_ROWS - i) != (MOE_MAX_EXPERT_ROWS - i + 127LL) / 128) ++bad;
    // sums of counts that no valid layout has: up to the end of an int and no further
    if (moe::sum_of(INT32_MAX - 3, 3) != INT32_MAX || moe::sum_of(INT32_MAX - 3, 5) != INT32_MAX ||
        moe::sum_of(INT32_MAX, INT32_MAX) != INT32_MAX || moe::sum_of(0, 0) != 0 || moe::sum_of(5, 7) != 12) ++bad;
    std::printf("%lld %lld\n", seen, bad);
    return bad != 0;
}
"""


def test_rows_of_tiles(tmp_path):
    from combine_moe_layout_04_gb300 import _build
    if not (os.path.exists("/usr/local/cuda/bin/nvcc") or shutil.which("nvcc")):
        pytest.skip("needs nvcc")
    src, exe = tmp_path / "rows.cu", tmp_path / "rows"
    src.write_text(PROGRAM)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", _build.CSRC, str(src), "-o",
                    str(exe), "-ldl"], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_more_rows_than_an_int_counts_are_refused():
    from combine_moe_layout_04_gb300 import _build
    _build.build()
    import combine_moe_layout_04_gb300 as moe
    from test_experts_refusals import GOOD, At, _lay, _refused
    lay, x = _lay(moe), moe.Experts(64, 64, GOOD, scales=GOOD)
    for T, k in ((2 ** 31 - 511, 1), (2 ** 31 - 1, 1), (2 ** 30 - 1, 2)):
        p = moe.Problem(T, 1024, k, 16, 1, 1)
        assert T * k > moe.MOE_MAX_EXPERT_ROWS
        codes = At(0x30000, (T * k, 32))
        for call, args in ((moe.moe_expert_forward, (lay, x, GOOD, GOOD)), (moe.moe_expert_backward_rows, (lay, x, GOOD, GOOD)),
                           (moe.moe_expert_backward_weights, (lay, x, GOOD, GOOD, GOOD)),
                           (moe.moe_expert_forward4, (lay, x, GOOD, GOOD, GOOD)), (moe.moe_quant4_rows, (lay, GOOD, codes, GOOD))):
            _refused(moe, moe.MOE_ERR_INVALID, call, p, *args)
        with pytest.raises(moe.MoeError):
            moe.moe_quant4_row_scale_bytes(p, 64)
    at_most = moe.Problem(moe.MOE_MAX_EXPERT_ROWS, 1024, 1, 16, 1, 1)
    assert moe.moe_quant4_row_scale_bytes(at_most, 64) == (moe.MOE_MAX_EXPERT_ROWS // 128 + 16) * 512
