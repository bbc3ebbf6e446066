"""Sanitizer build (CPU only) of the row operators' entry points: their
validation, sizes and overlap checks under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/csrc/row_ops_sanitize_main.c)."""
import os

import pytest

from qlora_fine_tuning_blockwise_amd import build as libbuild
from test_row_ops_sanitize import CSRC, ENV, ROOT, SAN, _run

HOST_SOURCES = ["rows_api.cpp", "embed.hip", "norm.hip", "distill.hip"]


def test_row_operator_entries_under_asan_ubsan(tmp_path):
    clang = "/opt/rocm/llvm/bin/clang"
    if not os.path.exists(clang):
        pytest.skip("ROCm clang not found")
    objdir = os.path.join(libbuild.PKG, "_build")
    others = [os.path.join(objdir, os.path.splitext(s)[0] + ".o") for s in libbuild.SOURCES
              if s not in HOST_SOURCES]
    if not all(os.path.exists(o) for o in others):
        libbuild.build()
    flags = [f for f in libbuild.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    for f in SAN:
        flags += ["-Xarch_host", f]
    objs = []
    for src in HOST_SOURCES:
        obj = str(tmp_path / (os.path.splitext(src)[0] + ".o"))
        _run([libbuild.hipcc(), *flags, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
    main = str(tmp_path / "main.o")
    _run([clang, "-std=c11", "-O1", "-g", *SAN, "-c",
          os.path.join(ROOT, "tests", "csrc", "row_ops_sanitize_main.c"), "-o", main])
    exe = str(tmp_path / "row_entries_san")
    _run([clang + "++", *SAN, main, *objs, *others, "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib",
          "-lamdhip64", "-o", exe])
    assert "every status as documented" in _run([exe], env=ENV)
