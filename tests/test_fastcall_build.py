"""The C++ marshalling is an addition: where it cannot be compiled the build goes
on without it, and one built for another interpreter or torch is not loaded."""
import os
import subprocess
import sys

import pytest
import torch

import __graft_entry__ as entry
from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U


@pytest.mark.parametrize("cxx", ["/bin/false", "/no/such/compiler"])
def test_a_failing_compiler_leaves_none_and_says_so(monkeypatch, tmp_path, capsys, cxx):
    path = tmp_path / "m.so"
    path.write_text("left from an earlier build")
    monkeypatch.setenv("CXX", cxx)
    monkeypatch.setattr(B, "fastcall_path", lambda: str(path))
    assert B.try_build_fastcall(force=True) is None
    assert not path.exists() and "no C++ marshalling" in capsys.readouterr().err
    with pytest.raises(RuntimeError, match="compiling"):
        B.build_fastcall(force=True)


def test_the_build_goes_on_without_it(monkeypatch, tmp_path):
    B.build()
    built = []
    monkeypatch.setenv("CXX", "/bin/false")
    monkeypatch.setattr(B, "fastcall_path", lambda: str(tmp_path / "m.so"))
    monkeypatch.setattr(B, "build", lambda **k: built.append(k))
    entry.build()
    assert len(built) == 2


def test_its_name_is_of_this_interpreter_and_torch(monkeypatch):
    assert torch.__version__ in os.path.basename(B.fastcall_path())
    assert sys.implementation.cache_tag in os.path.basename(B.fastcall_path())
    here = B.fastcall_path()
    monkeypatch.setattr(torch, "__version__", "1.0.other")
    assert B.fastcall_path() != here


def test_another_one_is_not_loaded(monkeypatch, tmp_path):
    """Where only a module of another name lies in the package nothing is bound."""
    B.build()
    (tmp_path / "_fastcall.so").write_bytes(b"")
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(U, "_fast", None)
    U._bind_fast(U.lib())
    assert U._fast is None
    (tmp_path / os.path.basename(B.fastcall_path())).write_bytes(b"no module")
    U._bind_fast(U.lib())
    assert U._fast is None


def test_the_one_of_this_torch_is_loaded_and_leaves_host_tensors_to_python():
    code = """
import torch
from long_context_sequence_seq_gb300 import build as B, ulysses as U
B.build(); B.build_fastcall(); U.lib()
assert U._fast is not None
t = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
inv, axes = U.rope_frequencies(128)
assert U._fast.rope(False, t, None, torch.zeros(4, dtype=torch.int32), inv, axes, "seq", "half", None, None) is None
kc, vc = torch.zeros(4, 2, 16, 128), torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
i = torch.zeros(4, 1, dtype=torch.int32)
assert U._fast.cache_write(t, t, kc, vc, i, i[:, 0], None, None, None, "seq") is None
for call in (lambda: U.cache_write(t, t, kc, vc, i, i[:, 0].contiguous()),
             lambda: U.cache_read(kc, vc, i, torch.zeros(5, dtype=torch.int32), 4),
             lambda: U.attn_decode(t, kc, vc, i, i[:, 0].contiguous())):
    try:
        call()
    except ValueError as e:
        assert "one shape and dtype" in str(e)
    else:
        raise AssertionError
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
