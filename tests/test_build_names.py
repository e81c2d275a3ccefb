"""The library's bytes depend on the sources alone: objects are named without
the temporary folder they are built in, whose path would get into them (and
measurements that are kept by the library's hash would be lost with every build)."""

import os

from agent_handoff_amd import build


def test_objects_have_the_same_names_in_every_build(monkeypatch):
    seen = []

    class Done:
        returncode, stderr, stdout = 0, "", ""

    def run(cmd, cwd=None, **_):
        seen.append((cmd, cwd))
        return Done

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    build.build()
    objects = [(cmd, cwd) for cmd, cwd in seen if "-c" in cmd]
    assert len(objects) == len(build.sources())
    for cmd, cwd in seen:
        assert cwd is None or not any(cwd in a for a in cmd)
    for cmd, cwd in objects:
        out = cmd[cmd.index("-o") + 1]
        assert cwd and not os.path.isabs(out)
