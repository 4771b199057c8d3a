"""Sanitizer tier (CPU only) of the decoder-block operators: 100000 seeded calls
with tensors laid out apart, in any order of dimensions, all of which must reach
their launcher; what the launchers are handed and the launch grids are checked
(tests/native/block_layout_san.cpp)."""

import os

from test_block_host_sanitizers import CLANGXX, ENV, HIPCC, PKG, ROOT, SAN, _run


def test_block_layouts_under_sanitizers(tmp_path):
    include = []
    for d in (os.path.join(ROOT, "include"), os.path.join(PKG, "csrc"), os.path.join(PKG, "csrc_block")):
        include += ["-I", d]
    objs = []
    for src in (os.path.join(PKG, "csrc_block", "block_api.hip"),
                os.path.join(ROOT, "tests", "native", "block_layout_san.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, "-x", "hip", "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
              "-Xarch_host", SAN[0], "-Xarch_host", SAN[1], "-Xarch_host", SAN[2], *include, "-c",
              src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "block_layout_san")
    _run([CLANGXX, *SAN, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    r = _run([exe], env=ENV, timeout=600)
    assert r.stdout == "ok 100000\n", r.stdout
