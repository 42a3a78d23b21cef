"""The choice of a kernel by a row's 32-column steps: every number up to the
largest dim's calls its own, any other is refused (needs a host compiler)."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

INCLUDES = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "fp8_prefill_gemm_amd", "csrc")]
SOURCE = r"""
#include <stdio.h>
#include <initializer_list>
#include "kv_steps.h"
int main() {
    for (unsigned c : {0u, 1u, 2u, 7u, 15u, 16u, 17u, 31u, 1u << 31, 0xFFFFFFFFu}) {
        int called = 0;
        const bool known = rz::with_steps(c, [&](auto n) { called = n; });
        printf("%u %d %d\n", c, known ? 1 : 0, called);
    }
}
"""


def test_with_steps(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    src, exe = tmp_path / "steps.cpp", tmp_path / "steps"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", *INCLUDES, str(src), "-o", str(exe)], check=True)
    got = [tuple(map(int, line.split())) for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert got == [(c, 1, c) if 1 <= c <= 16 else (c, 0, 0) for c in (0, 1, 2, 7, 15, 16, 17, 31, 1 << 31, 0xFFFFFFFF)]


def test_refusal_must_be_heeded(tmp_path):
    """A launcher that drops the answer draws a warning."""
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    src = tmp_path / "dropped.cpp"
    src.write_text('#include "kv_steps.h"\nint main() { rz::with_steps(3, [](auto) {}); }\n')
    done = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsyntax-only", *INCLUDES, str(src)], capture_output=True, text=True)
    assert done.returncode != 0 and "with_steps" in done.stderr
