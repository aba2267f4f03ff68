"""The binding module is rebuilt when the torch or Python it was built against is another one."""

import pytest


@pytest.fixture(scope="module")
def buildlib():
    import engram_gram_hash_gb300 as eg
    from engram_gram_hash_gb300 import buildlib

    eg.build()
    return buildlib


def test_step_module_follows_torch(buildlib, tmp_path, monkeypatch):
    assert not buildlib.step_stale()
    import torch

    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert buildlib.step_stale()
    monkeypatch.undo()
    assert not buildlib.step_stale()
    monkeypatch.setattr(buildlib, "STEP_STAMP", str(tmp_path / "none"))  # built before it was recorded
    assert buildlib.step_stale()


def test_only_what_is_stale_is_compiled(buildlib, tmp_path, monkeypatch):
    commands = []

    class Done:
        def __init__(self, cmd):
            commands.append(cmd)

        def wait(self):
            return 0

    monkeypatch.setattr(buildlib.subprocess, "Popen", Done)
    buildlib.build()
    assert not commands
    monkeypatch.setattr(buildlib, "STEP_STAMP", str(tmp_path / "stamp"))
    buildlib.build()
    assert len(commands) == 1 and buildlib.STEP_SRC in commands[0]
    buildlib.build()  # recorded
    assert len(commands) == 1
