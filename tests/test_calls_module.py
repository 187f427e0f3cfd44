"""The module of the attention block's calls: built for one torch, and needed by those calls alone."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def build():
    import __graft_entry__
    b = __graft_entry__._builder()
    b.build()
    return b


def run(code):
    return subprocess.run([sys.executable, "-c", "import sys; sys.path.insert(0, %r)\n" % ROOT + code], cwd="/",
                          capture_output=True, text=True, timeout=300)


def test_the_rest_does_without_it(build):
    """Imported, and its other calls made, where the module cannot be loaded; the attention block's calls say why."""
    r = run("""
class No:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._calls"):
            raise ImportError("no such module here")
sys.meta_path.insert(0, No())
import torch
import block_scaled_fp8_x128_gb300 as r9q
print(r9q.r9q_workspace_bytes(r9q.R9Q_OP_GEMM_W8A8, 64, 4096, 1024) > 0, r9q.r9q_strerror(0))
for _ in range(2):
    try:
        r9q._calls.kv4_gather
    except ImportError as e:
        print(e)
""")
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("True") and r.stdout.count("no such module here") == 2


def test_one_of_another_torch_is_refused(build):
    r = run("""
import torch
import block_scaled_fp8_x128_gb300 as r9q
torch.__version__ = "0.1"
for _ in range(2):
    try:
        r9q._calls.kv4_gather
        print("loaded")
    except ImportError as e:
        print(e)
""")
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("this is 0.1") == 2 and "loaded" not in r.stdout


def test_it_is_built_again_for_another_torch(build, tmp_path, monkeypatch):
    record = tmp_path / "for"
    assert build._other_than(str(record), build._built_for())
    record.write_text(build._built_for())
    assert not build._other_than(str(record), build._built_for())
    monkeypatch.setattr(build, "_torch_version", lambda: "0.1")
    assert build._other_than(str(record), build._built_for())


def test_it_names_the_torch_that_it_was_built_for(build):
    import torch
    import block_scaled_fp8_x128_gb300 as r9q
    assert callable(r9q._calls.kv4_gather) and r9q._calls.torch_version == torch.__version__ == build._torch_version()
