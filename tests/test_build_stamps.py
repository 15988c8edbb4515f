"""What makes a built library out of date (no GPU, nothing is compiled)."""
import sys

import torch

from scaled_dot_product_bwd_b200 import build


def test_the_marshalling_module_is_rebuilt_for_another_torch_or_python(monkeypatch):
    flags = ["-O2"]
    first = build._bind_stamp(flags)
    assert build._bind_stamp(flags) == first and build._bind_stamp(["-O1"]) != first
    for owner, name, value in ((torch, "__version__", "2.99.0"), (torch.version, "git_version", "0" * 40),
                               (sys, "version", "3.99.0 (main)")):
        with monkeypatch.context() as m:
            m.setattr(owner, name, value)
            assert build._bind_stamp(flags) != first, name
    assert build._bind_stamp(flags) == first


def test_a_stamp_of_other_sources_or_flags_runs_the_compiler(monkeypatch, tmp_path):
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done()

    monkeypatch.setattr(build.subprocess, "run", run)
    out = str(tmp_path / "lib.so")
    build._make(out, "a", ["cc"], False, False)
    build._make(out, "a", ["cc"], False, False)
    assert len(ran) == 1
    build._make(out, "b", ["cc"], False, False)
    build._make(out, "b", ["cc"], False, True)
    assert len(ran) == 3
