"""Tests that hand made-up device addresses to the C entry points run on hosts
without a GPU alone, where a check that goes missing cannot launch a kernel on
them: each such test is marked so, or is one that the collection marks."""

import ast
import os

import conftest

HERE = os.path.dirname(os.path.abspath(__file__))
CALLS = {"test_attend_abi_host.py": {"_rotate", "_copy", "_attend", "_pool"},
         "test_attend_limits_host.py": {"_rotate", "_in_place", "_read"}, "test_attend_workspace.py": {"kvpage_attend"}}


def _callers(name):
    """Tests of a file that make such calls, and whether they are decorated."""
    with open(os.path.join(HERE, name)) as f:
        tree = ast.parse(f.read())
    for fn in tree.body:
        if isinstance(fn, ast.FunctionDef) and fn.name.startswith("test"):
            called = {getattr(c.func, "id", getattr(c.func, "attr", "")) for c in ast.walk(fn) if isinstance(c, ast.Call)}
            raw = "kvpage_attend" not in CALLS[name] or "L" in {n.id for n in ast.walk(fn) if isinstance(n, ast.Name)}
            if called & CALLS[name] and raw:
                yield fn.name, any(getattr(d, "id", "") == "fake_addresses" for d in fn.decorator_list)


def test_every_such_test_is_left_out_where_there_is_a_gpu():
    seen = 0
    for name in CALLS:
        for test, marked in _callers(name):
            seen += 1
            assert marked or (name, test) in conftest.FAKE_ADDRESSES, (name, test)
    assert seen >= 9


class _Item:
    def __init__(self, file, name):
        self.path, self.originalname, self.marks = type("P", (), {"name": file}), name, []

    def add_marker(self, mark):
        self.marks.append(mark)


def test_the_collection_marks_them(monkeypatch):
    for count in (0, 1):
        monkeypatch.setattr(conftest, "_gpus", lambda: count)
        items = [_Item(f, n) for f, n in sorted(conftest.FAKE_ADDRESSES)] + [_Item("test_abi_host.py", "test_other")]
        conftest.pytest_collection_modifyitems(items)
        assert [len(i.marks) for i in items] == [count] * (len(items) - 1) + [0]
        assert all(m.name == "skip" for i in items for m in i.marks)
