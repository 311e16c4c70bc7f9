"""What importing the package loads: neither torch nor a library, by any form of import; the names of the 4-bit operands and
the expert layer, listed by dir(), load theirs at their first use."""
import os
import subprocess
import sys

import block_quantized_weight_pn3t_gb300 as pnq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def loaded_after(statement):
    """Of torch and the package's libraries, what a fresh interpreter has loaded after a statement."""
    code = f"""
import sys
{statement}
maps = open("/proc/self/maps").read()
print([n for n, there in (("torch", "torch" in sys.modules), ("libpnq.so", "libpnq.so" in maps), ("_native.so", "_native.so" in maps)) if there])
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout.strip()


def test_imports_load_nothing():
    name = pnq.__name__
    assert loaded_after(f"import {name}") == "[]"
    assert loaded_after(f"from {name} import *\ngemv, PnqError, NVFP4") == "[]"
    assert loaded_after(f"import {name} as p\ndir(p)") == "[]"


def test_lazy_names():
    listed = dir(pnq)
    for n in pnq._FP4_NAMES:
        assert n in listed and n not in pnq.__all__
    for n in pnq.__all__:
        assert n in listed and hasattr(pnq, n)
    assert not hasattr(pnq, "no_such_name")
