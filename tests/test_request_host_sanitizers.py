"""Sanitizer tier (CPU only) of the operators on requests of many lengths: the C
entry points, built with AddressSanitizer and UndefinedBehaviorSanitizer on the
host side, over 200000 seeded calls with the launchers replaced by checks of
what the planners hand to the kernels (tests/native/request_san.cpp)."""

import os

from test_block_host_sanitizers import CLANGXX, ENV, HIPCC, PKG, ROOT, SAN, _run


def test_request_entry_points_under_sanitizers(tmp_path):
    include = []
    for d in (os.path.join(ROOT, "include"), os.path.join(PKG, "csrc"), os.path.join(PKG, "csrc_block")):
        include += ["-I", d]
    objs = []
    for src in (os.path.join(PKG, "csrc_block", "request_api.hip"),
                os.path.join(ROOT, "tests", "native", "request_san.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        # sanitizers on the host side only; no device code is built into these
        _run([HIPCC, "-x", "hip", "-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
              "-Xarch_host", SAN[0], "-Xarch_host", SAN[1], "-Xarch_host", SAN[2], *include, "-c",
              src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "request_san")
    _run([CLANGXX, *SAN, *objs, "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    r = _run([exe], env=ENV, timeout=600)
    assert r.stdout.startswith("ok "), r.stdout
    assert int(r.stdout.split()[1]) > 20000, r.stdout  # enough of the shapes reached a launch
