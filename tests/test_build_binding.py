"""The binding is linked anew for the torch and Python it is loaded into, whatever was built in between."""
import subprocess
import sysconfig

import pytest
import torch

import greedy_decode_step_gb300  # noqa: F401



@pytest.fixture
def builder(monkeypatch, tmp_path):
    """build() over a folder of its own, with a compiler that only writes its output file."""
    import sys
    mod = sys.modules["greedy_decode_step_gb300.build"]
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "libdec.so"))
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(mod, "UNITS", [])
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("\n".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mod.subprocess, "run", run)

    def build():
        commands.clear()
        mod.build()
        with open(mod.BINDING) as f:
            return [a for a in f.read().split("\n") if a.endswith(".o")], len(commands)

    return build


@pytest.mark.parametrize("what", ["torch", "python"])
def test_the_binding_follows_the_versions(builder, monkeypatch, what):
    abi = sysconfig.get_config_var

    def use(v):
        if what == "torch":
            monkeypatch.setattr(torch, "__version__", v)
        else:
            monkeypatch.setattr(sysconfig, "get_config_var", lambda n: v if n in ("SOABI", "EXT_SUFFIX") else abi(n))

    use("one")
    first, _ = builder()
    use("two")
    second, _ = builder()
    assert first != second
    use("one")
    assert builder()[0] == first
    assert builder() == (first, 0)  # and nothing to do the second time
