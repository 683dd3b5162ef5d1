"""A package whose native module is not built says what to build, as for the library itself."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "selective_state_update_amd"


@pytest.mark.parametrize("missing", ["_native.so", "libssu.so"])
def test_missing_library(tmp_path, missing):
    there = tmp_path / PACKAGE
    there.mkdir()
    shutil.copy(os.path.join(ROOT, PACKAGE, "__init__.py"), there)
    for name in {"_native.so", "libssu.so"} - {missing}:
        os.symlink(os.path.join(ROOT, PACKAGE, name), there / name)
    r = subprocess.run([sys.executable, "-c", f"import {PACKAGE}"], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode != 0
    last = r.stderr.strip().splitlines()[-1]
    assert last.startswith("ImportError: ") and missing in last and "is not built" in last and "build.py" in last, r.stderr
