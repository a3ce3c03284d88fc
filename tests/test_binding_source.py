"""The binding's source: no function of a module is defined twice (the first would never run)."""
import ast
import pathlib

import pytest

import rwkv_linear_attention_gb300 as wkv7

FILES = sorted(pathlib.Path(wkv7.__file__).parent.glob("*.py"))


@pytest.mark.parametrize("path", FILES, ids=lambda p: p.name)
def test_no_name_is_defined_twice(path):
    tree = ast.parse(path.read_text())
    scopes = [tree.body] + [n.body for n in ast.walk(tree) if isinstance(n, ast.ClassDef)]
    for body in scopes:
        names = [n.name for n in body if isinstance(n, (ast.FunctionDef, ast.AsyncFunctionDef, ast.ClassDef))]
        assert sorted(names) == sorted(set(names))


def test_every_public_name_exists():
    assert len(set(wkv7.__all__)) == len(wkv7.__all__)
    for name in wkv7.__all__:
        assert hasattr(wkv7, name), name
