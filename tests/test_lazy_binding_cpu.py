"""The compiled calls are names of the package without their library; the first call loads it."""
import inspect
import os
import subprocess
import sys

import pytest

import optimizer_fp8_cast_b200 as fp8
from optimizer_fp8_cast_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = ("fp8_rmsnorm_cast", "fp8_rmsnorm_backward", "fp4_cast_multi", "fp4_gemm_multi")
# a package whose libraries are not built
UNBUILT = ("import optimizer_fp8_cast_b200 as p; p.LIB_PATH = p.BINDING_PATH = '/nonexistent/lib.so';"
           "assert p._lib is None;")


def run(code):
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)


def test_names_need_no_library():
    run(UNBUILT + "from optimizer_fp8_cast_b200 import *;"
        f"assert all(hasattr(p, n) and callable(globals()[n]) for n in {CALLS});"
        "import inspect; assert 'workspace' in inspect.signature(fp8_rmsnorm_backward).parameters; assert p._lib is None")


@pytest.mark.parametrize("name", CALLS)
def test_a_call_without_the_library_raises(name):
    run(UNBUILT + f"""
try:
    p.{name}([])
except RuntimeError as e:
    assert 'not built' in str(e)
else:
    raise AssertionError('no error')
""")


def test_first_call_puts_the_compiled_functions_in_the_package():
    build.build()
    run("""
import optimizer_fp8_cast_b200 as p
held = p.fp4_gemm_multi
for call in (p.fp4_cast_multi, held, p.fp4_gemm_multi):
    try:
        call(1)
    except TypeError as e:
        assert 'must be a list of dicts' in str(e)
assert all(type(getattr(p, n)).__name__ == 'builtin_function_or_method' for n in %r)
""" % (CALLS,))


@pytest.mark.parametrize("name", CALLS)
def test_declaration_and_compiled_function_say_the_same(name):
    build.build()
    code = f"import inspect, optimizer_fp8_cast_b200 as p; f = p.{name}; print(inspect.signature(f), inspect.getdoc(f))"
    declared = subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, capture_output=True, text=True).stdout
    compiled = getattr(fp8._load_binding(), name)
    assert declared == f"{inspect.signature(compiled)} {inspect.getdoc(compiled)}\n"
