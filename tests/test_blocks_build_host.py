"""The library builds and is called where the compiled binding, or torch, is missing."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, text=True, stdout=subprocess.PIPE,
                          stderr=subprocess.STDOUT, timeout=600)


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def test_the_library_builds_without_torch():
    r = run("import sys, runpy; sys.modules['torch'] = None\n"
            "m = runpy.run_path('int8_kv_decode_gb300/build.py')\n"
            "print(m['build']())")
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip().endswith("libkattn.so")


def test_a_binding_that_does_not_compile_leaves_the_library(tmp_path):
    # the library is linked all the same, the error is raised, and no older binding is left
    r = run(f"import os, shutil, runpy; p = {str(tmp_path)!r}\n"
            "for d in ('include', 'int8_kv_decode_gb300'):\n"
            "    shutil.copytree(d, os.path.join(p, d), copy_function=shutil.copy2)\n"
            "q = os.path.join(p, 'int8_kv_decode_gb300')\n"
            "os.remove(os.path.join(q, 'libkattn.so'))\n"
            "open(os.path.join(q, 'csrc', 'bind.cpp'), 'a').write('#error no')\n"
            "m = runpy.run_path(os.path.join(q, 'build.py'))\n"
            "try:\n"
            "    m['build']()\n"
            "except RuntimeError as e:\n"
            "    print('raised' if 'bind.cpp' in str(e) else e)\n"
            "print(os.path.exists(os.path.join(q, 'libkattn.so')), os.path.exists(os.path.join(q, '_bind.so')))\n")
    assert r.returncode == 0, r.stdout
    assert r.stdout.split() == ["raised", "True", "False"], r.stdout


HIDDEN = ("import sys; sys.modules['int8_kv_decode_gb300._bind'] = None\n"
          "import warnings, torch, int8_kv_decode_gb300 as K\n")


def test_calls_are_checked_without_the_binding():
    # the refusals of api.py, and one warning for the whole process
    r = run(HIDDEN + "x, i = torch.zeros(2, 3, 128), torch.zeros(2, dtype=torch.int32)\n"
            "with warnings.catch_warnings(record=True) as w:\n"
            "    warnings.simplefilter('always')\n"
            "    for _ in range(2):\n"
            "        try:\n"
            "            K.rope(x, i, torch.zeros(5, 64, 2), out=x)\n"
            "        except ValueError as e:\n"
            "            print('refused:', e)\n"
            "print([(m.category.__name__, 'binding' in str(m.message)) for m in w])\n")
    assert r.returncode == 0, r.stdout
    assert r.stdout.count("refused:") == 2, r.stdout
    assert "[('RuntimeWarning', True)]" in r.stdout, r.stdout


def test_a_binding_of_another_torch_is_not_used():
    r = run("import torch, warnings\n"
            "from int8_kv_decode_gb300 import _bind, api\n"
            "assert _bind.torch_version == torch.__version__\n"
            "torch.__version__ = '0.0'\n"
            "with warnings.catch_warnings(record=True) as w:\n"
            "    warnings.simplefilter('always')\n"
            "    print(api._load_plain() is _bind, len(w))\n")
    assert r.returncode == 0, r.stdout
    assert r.stdout.strip().endswith("False 1"), r.stdout
