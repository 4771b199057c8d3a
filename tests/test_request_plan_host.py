"""Host-only checks of what a chunk call's sizes make of it: the kernel, its splits and
its workgroups, read from what the entry point hands to the launchers
(tests/native/request_plan.cpp)."""

import os
import subprocess

import pytest

import request_cases as cases
from test_block_host_sanitizers import CLANGXX, HIPCC, PKG, ROOT, _run
from vision_upsampler_decoders_amd import ctconv as C

F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(B, rows, n, Hq, Hkv, D, max_length, window, weights, dtype, packed) ->
    (kernel, splits, keys per split, workgroups)."""
    tmp = tmp_path_factory.mktemp("plan")
    include = []
    for d in (os.path.join(ROOT, "include"), os.path.join(PKG, "csrc"), os.path.join(PKG, "csrc_block")):
        include += ["-I", d]
    objs = []
    for src in (os.path.join(PKG, "csrc_block", "request_api.hip"),
                os.path.join(ROOT, "tests", "native", "request_plan.cpp")):
        objs.append(str(tmp / (os.path.basename(src) + ".o")))
        _run([HIPCC, "-x", "hip", "-O1", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
              "--offload-host-only", *include, "-c", src, "-o", objs[-1]])
    exe = str(tmp / "request_plan")
    _run([CLANGXX, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])

    def ask(*sizes, packed=1):
        line = " ".join(str(int(v)) for v in (*sizes, packed)) + "\n"
        r = subprocess.run([exe], input=line, capture_output=True, text=True, check=True)
        kernel, splits, chunk, groups = r.stdout.split()
        return kernel, int(splits), int(chunk), int(groups)

    return ask


@pytest.mark.parametrize("dt", [F32, BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,rows", [(1, 1), (4, 4), (3, 40), (48, 48)])
def test_a_bound_on_the_rows_past_their_number_changes_nothing(plan, B, rows, D, dt):
    """No sequence has more rows than the call: n = 2048 and 16384 plan as n = rows does."""
    want = plan(B, rows, rows, 8, 8, D, 131072, 0, 0, dt)
    for n in (rows + 1, 2048, 16384):
        assert plan(B, rows, n, 8, 8, D, 131072, 0, 0, dt) == want, n
        for weights in (False, True):
            f = C.ctconv_chunk_attention_workspace_bytes
            assert (f(B, rows, n, 8, 8, D, 131072, 0, weights, dt) ==
                    f(B, rows, rows, 8, 8, D, 131072, 0, weights, dt))
    if B < 48:  # few workgroups over many keys: divided
        assert want[1] > 16


@pytest.mark.parametrize("dt,D", [(F32, 64), (F32, 256), (BF16, 64)])
def test_workgroups_without_rows_do_not_stop_a_split(plan, dt, D):
    """One sequence with many rows among single ones: in the streaming kernel most workgroups of
    the grid have no rows, and those that have are too few to walk 60000 keys whole."""
    B, n = 24, 128
    kernel, splits, _, groups = plan(B, B - 1 + n, n, 12, 12, D, 60000, 0, 0, dt)
    assert kernel == "tile" or (splits >= 4 and groups < 1 << 20)


CODE = {"f32": F32, "bf16": BF16, "f16": F16}


@pytest.mark.parametrize("case", cases.ODD, ids=[str(i) for i in range(len(cases.ODD))])
def test_cases_of_odd_values_reach_their_kernel(plan, case):
    dt, counts, lengths, H, G, D, window, kernel, split = case
    got = plan(len(counts), sum(counts), max(counts), H * G, H, D, max(lengths), window, 0, CODE[dt])
    assert got[0] == kernel and (got[1] > 1) == split, got
    if kernel == "stream" and not split and max(lengths) > 1024:
        assert got[2] > 1024  # its places are staged more than once


def test_tiled_cases_reach_the_tiled_kernel(plan):
    for dt, (counts, lengths, n, Hq, H, D, page, window, _) in cases.TILED:
        most = (-(-max(lengths) // page) + 1) * page
        for weights in (0, 1):
            assert plan(len(counts), sum(counts) + 3, n, Hq, H, D, most, window, weights,
                        CODE[dt])[0] == "tile", (counts, D)
            assert plan(len(counts), len(counts) * n, n, Hq, H, D, most, window, weights, CODE[dt],
                        packed=0)[0] == "tile", (counts, D)
    for dt, (counts, lengths, n, Hq, H, D, page, window, _) in cases.NARROW:
        most = (-(-max(lengths) // page) + 1) * page
        assert plan(len(counts), sum(counts) + 3, n, Hq, H, D, most, window, 1,
                    CODE[dt])[0] == "tile", (counts, D)
    for dt, n, Hq, H, D in cases.CUT:
        most = -(-(n + 900) // 16) * 16
        assert plan(2, 2 * n - 1 - n // 2, n, Hq, H, D, most, 0, 1, CODE[dt])[0] == "tile"
    for dt, n, Hq, H, extra in cases.MISSING:
        for most in (160 + extra, 150 + extra):
            assert plan(5, 5 * n, n, Hq, H, 64, most, 0, 1, CODE[dt], packed=0)[0] == "tile"


def test_page_0_case_reaches_the_tiled_kernel(plan):
    assert plan(2, 256, 128, 32, 8, 128, 8000, 0, 0, BF16)[0] == "tile"
