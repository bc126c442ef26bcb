"""One library a process (no GPU): the compiled binding uses the one that
FP8LIN_LIB names, and one that is too old or too new is refused by name."""
import os
import shutil
import subprocess
import sys

import pytest

from tensor_scaled_fp8_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OWN = os.path.join(ROOT, "tensor_scaled_fp8_amd", "lib", "libfp8lin.so")


def _python(code, lib):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, env={**os.environ, "FP8LIN_LIB": str(lib)},
                          capture_output=True, text=True, timeout=300)


def test_the_binding_uses_the_named_library(tmp_path):
    other = tmp_path / "libfp8lin.so"
    shutil.copy(OWN, other)
    r = _python("from tensor_scaled_fp8_amd import block\n"
                "block._binding()\n"
                "print(sorted({l.split()[-1] for l in open('/proc/self/maps') if 'libfp8lin' in l}))", other)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str([str(other)])


def _library(tmp_path, source):
    c, so = tmp_path / "lib.c", tmp_path / "libfp8lin.so"
    c.write_text(source)
    subprocess.run(["gcc", "-shared", "-fPIC", str(c), "-o", str(so)], check=True)
    return so


@pytest.mark.parametrize("source,said", [
    (f"int fp8_abi_version(void) {{ return {_lib.ABI_VERSION}; }}", "lacks fp8_"),
    (f"int fp8_abi_version(void) {{ return {_lib.ABI_VERSION - 1}; }}", f"ABI {_lib.ABI_VERSION - 1} != expected"),
    ("int unrelated(void) { return 0; }", "ABI unknown != expected")])
def test_another_library_is_refused(tmp_path, source, said):
    r = _python("import tensor_scaled_fp8_amd as t\nt.load()", _library(tmp_path, source))
    assert r.returncode == 1 and "ImportError" in r.stderr and said in r.stderr, r.stderr
