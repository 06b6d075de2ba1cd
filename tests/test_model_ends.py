"""The operators at a model's two ends together, and the host-side agreement of
include/flce_model.h with its binding."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header():
    with open(os.path.join(ROOT, "include", "flce_model.h")) as f:
        return re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)


def test_header_matches_binding():
    from linear_cross_entropy_02_gb300 import _lib
    names = sorted(set(re.findall(r"\b(flce_[a-z_]+)\s*\(", header())))
    assert sorted(_lib.MODEL_EXPORTED) == names
    for name, args in re.findall(r"\b(flce_[a-z_]+)\s*\(([^)]*)\)\s*;", header()):
        assert len(getattr(_lib.lib(), name).argtypes) == args.count(",") + 1, name
    for name, val in re.findall(r"#define (FLCE_[A-Z0-9_]+) (\d+)", header()):
        assert getattr(_lib, name) == int(val), name


def test_kernel_names():
    from linear_cross_entropy_02_gb300 import _lib as B
    first, n = B.FLCE_MODEL_KERNEL_FIRST, B.FLCE_MODEL_KERNEL_COUNT
    names = [B.lib().flce_kernel_name(i).decode() for i in range(first, first + n)]
    assert len(set(names)) == n and "unknown" not in names
    assert B.lib().flce_kernel_name(first - 1) == B.lib().flce_kernel_name(first + n) == b"unknown"


def test_header_is_plain_c(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "flce_model.h"\nint main(void) { return flce_embedding == 0; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-Wno-address", "-I", os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
