"""The INT4 calls run the library of their own package, wherever that package was copied to."""
import os
import shutil
import subprocess
import sys
import threading
import time

import pytest

from bit_kv_cache_oscar_gb300 import binding as ob
from bit_kv_cache_oscar_gb300 import build

PKG = os.path.dirname(os.path.abspath(build.__file__))
ROOT = os.path.dirname(PKG)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def run(code, root):
    p = subprocess.run([sys.executable, "-c", code], cwd=root, env={**os.environ, "PYTHONPATH": str(root)}, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
    return p.stdout.split()


MAPPED = """
from bit_kv_cache_oscar_gb300 import binding as ob
ob._native()
print(*sorted({l.split()[-1] for l in open('/proc/self/maps') if l.rstrip().endswith(('liboscar.so', '_marshal.so'))}), sep='\\n')
"""


def copied(to):
    shutil.copytree(PKG, to / os.path.basename(PKG), ignore=shutil.ignore_patterns("__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), to / "include")
    return to


def test_a_copied_package_maps_its_own_library_alone(tmp_path):
    pkg = copied(tmp_path) / os.path.basename(PKG)
    assert run(MAPPED, tmp_path) == [str(pkg / "_marshal.so"), str(pkg / "liboscar.so")]


def test_a_moved_package_without_the_original(tmp_path):
    first, second = tmp_path / "first", tmp_path / "second"
    first.mkdir()
    copied(first)
    run("from bit_kv_cache_oscar_gb300 import build; build.build()", first)      # what depends on the place is made anew
    first.rename(second)
    pkg = second / os.path.basename(PKG)
    assert run(MAPPED, second) == [str(pkg / "_marshal.so"), str(pkg / "liboscar.so")]


def test_what_was_made_with_another_torch_is_made_again(tmp_path):
    code = """
import os, torch
from bit_kv_cache_oscar_gb300 import build
build.build()
out = os.path.join(build.BUILD, 'marshal.o')
before = os.path.getmtime(out)
build.build()
assert os.path.getmtime(out) == before
torch.__version__ += '.other'
build.build()
assert os.path.getmtime(out) > before
"""
    run(code, copied(tmp_path))


def test_threads_see_the_extension_only_when_it_is_complete(monkeypatch):
    from importlib.machinery import ExtensionFileLoader
    load = ExtensionFileLoader.exec_module

    def slow(self, module):
        time.sleep(0.2)
        load(self, module)

    monkeypatch.setattr(ExtensionFileLoader, "exec_module", slow)
    monkeypatch.setattr(ob, "_marshal", None)
    seen, gate = [], threading.Barrier(3)

    def work(wait):
        gate.wait()
        time.sleep(wait)
        ob._native()
        with pytest.raises(ob.OscarError):                # the refusals' class is known
            ob._native().promote_int4(ob.Layout(1, 1, 16), *[None] * 7)
        seen.append(wait)

    threads = [threading.Thread(target=work, args=(w,)) for w in (0, 0.05, 0.1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(seen) == 3
