"""The extension module that hands tensors to the short calls: built beside the library for one torch
and one Python, and needed by those calls alone. No test here needs a GPU."""
import os
import subprocess
import sys

import pytest
import torch

from paged_decode_attention_02_gb300 import binding, build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    build_lib.build()


_WITHOUT = """
import sys
sys.path.insert(0, {root!r})
import torch
from paged_decode_attention_02_gb300 import binding, build_lib
build_lib.marshal_path = lambda: {missing!r}
lib = binding.load()
assert binding.status_string(0) == "ok" and lib.pda_version() == 1
i = torch.zeros((1, 1), dtype=torch.int32)
try:
    binding.kv_assign_blocks(i, i[0], i[0], i[0], i[0], 16)
except ValueError:
    pass  # tensors of the host: refused by the call itself
else:
    raise SystemExit("not refused")
try:
    binding._load_marshal()
except RuntimeError as e:
    assert "extension module" in str(e) and {missing!r} in str(e)
else:
    raise SystemExit("no error")
"""


def test_the_librarys_other_calls_do_without_it(tmp_path):
    code = _WITHOUT.format(root=ROOT, missing=str(tmp_path / "none.so"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-2000:]


def test_it_is_loaded_once_and_names_the_calls():
    m = binding._load_marshal()
    assert m is binding._load_marshal()
    for name in ("qk_norm_rope_append", "qk_norm_rope", "paged_window_attention",
                 "paged_window_chunk_attention", "verify_drafts"):
        assert callable(getattr(m, name))


def test_another_torch_or_python_asks_for_another_file(monkeypatch):
    path = build_lib.marshal_path()
    assert os.path.exists(path) and build_lib.marshal_up_to_date()
    for obj, name, value in ((torch, "__version__", "9.9.9"),
                             (torch._C, "_GLIBCXX_USE_CXX11_ABI",
                              not torch._C._GLIBCXX_USE_CXX11_ABI),
                             (build_lib.sysconfig, "get_config_var", lambda _: ".cpython-399.so")):
        with monkeypatch.context() as m:
            m.setattr(obj, name, value)
            assert build_lib.marshal_path() != path
            assert not build_lib.marshal_up_to_date() and build_lib.up_to_date()
    assert build_lib.marshal_path() == path


def test_a_failing_host_compiler_leaves_the_library(monkeypatch, tmp_path):
    monkeypatch.setattr(build_lib, "marshal_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setenv("CXX", "/bin/false")
    t = os.path.getmtime(build_lib.LIB_PATH)
    with pytest.raises(RuntimeError, match="none.so"):
        build_lib.build()
    assert os.path.getmtime(build_lib.LIB_PATH) == t
