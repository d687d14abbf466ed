"""What build() makes of hosts and module files that are not as they should be."""
import os
import shutil
import sys

import pytest

from bit_decode_attention_b200 import _native
from bit_decode_attention_b200 import build as nvbuild


@pytest.fixture(autouse=True, scope="module")
def built():
    nvbuild.build()


def test_binding_says_what_it_was_built_for():
    assert nvbuild.binding_up_to_date()
    assert _native.binding().built_for == nvbuild.binding_stamp()


def test_binding_of_another_torch_is_built_again(monkeypatch, tmp_path):
    """File times alone say that a module built before a torch upgrade is up to date."""
    monkeypatch.setattr(nvbuild.subprocess, "run", lambda cmd, check: made.append(cmd) or shutil.copy(copy, out(cmd)))
    copy, made, out = str(tmp_path / "b.so"), [], lambda cmd: cmd[cmd.index("-o") + 1]
    shutil.copy(nvbuild.BINDING, copy)
    monkeypatch.setattr(nvbuild, "BINDING", str(tmp_path / "_binding.so"))
    assert not nvbuild.binding_up_to_date() and nvbuild.build_binding() and len(made) == 1
    assert nvbuild.build_binding() and len(made) == 1
    stamp = nvbuild.binding_stamp()
    for other in (stamp + "1", stamp[:-1], stamp.replace("torch ", "torch 1")):
        monkeypatch.setattr(nvbuild, "binding_stamp", lambda: other)
        assert not nvbuild.binding_up_to_date() and nvbuild.build_binding()
    assert len(made) == 4 and any(f.endswith('"%s"' % other) for f in made[-1])


@pytest.mark.parametrize("lacks", ["torch", "headers", "g++"])
def test_library_is_built_without_what_the_binding_needs(monkeypatch, capsys, lacks):
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif lacks == "headers":
        monkeypatch.setattr(nvbuild.sysconfig, "get_paths", lambda: {"include": os.path.join(nvbuild.HERE, "nothing")})
    else:
        monkeypatch.setattr(nvbuild.shutil, "which", lambda name: None)
    assert nvbuild.build() == nvbuild.LIB
    assert "_binding.so is not built" in capsys.readouterr().err
