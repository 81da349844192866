"""AddressSanitizer and UndefinedBehaviorSanitizer builds of the host code of the operators around an
expert sub-layer, on the CPU: argument checks, launch shapes and workspace sizes (``csrc/ffn_api.cpp``
and the host side of the operators' own sources), driven by ``tests/sanitize/sublayer_driver.cpp``; no
call reaches a GPU."""
from __future__ import annotations

import glob
import os
import subprocess

import pytest

from test_sanitizers import CSRC, HIPCC, ROOT, SAN, _run_clean

SOURCES = ("ffn_api.cpp", "ffn_noalloc.hip", "rmsnorm.hip", "moe_dispatch.hip", "ffn_q4.hip")


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_sublayer_entry_points_under_sanitizers(tmp_path):
    from transformer_ffn_fusion_amd import build as B
    objdir = os.path.join(ROOT, "transformer_ffn_fusion_amd", "_build")

    def built():
        return [o for o in glob.glob(os.path.join(objdir, "*.hip.o"))
                if os.path.basename(o)[:-2] not in SOURCES]
    if len(built()) < 5:
        B.build()
    flags = ["-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    for f in ("-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all"):
        flags += ["-Xarch_host", f]
    flags += ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    objs, running = [], []
    for src in [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(SAN, "sublayer_driver.cpp")]:
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        running.append(subprocess.Popen([HIPCC, *flags, "-c", src, "-o", objs[-1]], stdout=subprocess.DEVNULL,
                                        stderr=subprocess.DEVNULL))
    assert [r.wait() for r in running] == [0] * len(running)
    exe = str(tmp_path / "sublayer_san")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-Xarch_host", "-fsanitize=address",
                    "-Xarch_host", "-fsanitize=undefined", *objs, *built(), "-o", exe],
                   check=True, capture_output=True)
    assert "ok" in _run_clean(exe, {"ASAN_OPTIONS": "detect_leaks=0"})
