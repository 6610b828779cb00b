"""Which heads of a scan stay together on one XCD (csrc/lin_plan.hpp), compiled
for the host."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mamba_selective_ssm_ssd_amd", "csrc")


@pytest.fixture(scope="module")
def head_group(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    d = tmp_path_factory.mktemp("lin_plan")
    (d / "plan.cpp").write_text('#include "lin_plan.hpp"\nextern "C" int32_t head_group(int32_t share, int32_t heads, int64_t segments, '
                                'int32_t columns, int32_t scans, int32_t cut) {\n'
                                '    return m3::lin_head_group(share, heads, segments, columns, scans, cut != 0);\n}\n')
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"),
                    "-o", str(d / "plan.so")], check=True)
    f = ctypes.CDLL(str(d / "plan.so")).head_group
    f.argtypes, f.restype = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int64, *[ctypes.c_int32] * 3], ctypes.c_int32
    return f


def _busiest(hg, heads, segments, tiles):
    """Workgroups of the fullest XCD where groups go round the eight."""
    load = [0] * 8
    for g in range(segments * (heads // hg)):
        load[g % 8] += hg * tiles
    return max(load)


@pytest.mark.parametrize("share,heads,segments,columns,scans,cut", [
    (64, 64, 1, 4, 1, False), (64, 64, 1, 4, 3, False), (64, 64, 1, 1, 3, False), (64, 64, 5, 4, 1, True), (8, 32, 1, 2, 3, False),
    (8, 24, 1, 2, 3, False), (8, 24, 1, 4, 3, False), (12, 48, 3, 1, 1, False), (12, 48, 3, 1, 3, False), (7, 7, 1, 8, 3, False),
    (1, 64, 1, 4, 3, False), (1, 8, 17, 1, 3, False), (5, 40, 13, 1, 3, True), (30, 30, 2, 4, 1, False), (1000, 1000, 1, 4, 1, False)])
def test_groups_leave_no_xcd_idle(head_group, share, heads, segments, columns, scans, cut):
    hg, tiles = head_group(share, heads, segments, columns, scans, cut), columns * scans
    assert hg >= 1 and heads % hg == 0
    most, mean = _busiest(hg, heads, segments, tiles), segments * heads * tiles / 8
    assert most <= 32 or most <= 9 / 8 * mean or hg == 1, (hg, most, mean)


def test_groups_hold_the_heads_that_share_rows_where_there_are_enough(head_group):
    # 16 ragged sequences in segments, gradients of grouped heads, a short piece that fits four XCDs' units at once
    assert head_group(4, 32, 32, 1, 1, True) == 4 and head_group(8, 32, 16, 1, 3, True) == 8
    assert head_group(4, 16, 1, 4, 1, False) == 4
    # neighbours without a common row join only where many groups are left
    assert head_group(1, 64, 65, 1, 1, True) == 16 and head_group(1, 64, 4, 1, 3, False) == 8 and head_group(1, 32, 33, 1, 1, True) == 4
