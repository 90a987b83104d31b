"""A C program linked with the built library by its path starts wherever it is run."""
import os
import shutil
import subprocess

import pytest

import transformer_encoder_forward_gb300 as te
from tests.test_abi import L, ROOT  # noqa: F401  (the built library as a fixture)


def test_a_c_program_linked_by_path_runs(L, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "v.c", tmp_path / "v"
    src.write_text('#include <stdio.h>\n#include "tefwd.h"\nint main(void) { puts(te_version()); return 0; }\n')
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), te.LIB_PATH, "-o", str(exe)], check=True)
    env = {k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"}
    r = subprocess.run([str(exe)], cwd=tmp_path, env=env, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == te.version(), r.stderr
