"""The entry script: what it does when it is run, which an import does not show."""
import ast
import os

from conftest import ROOT


def test_everything_is_defined_before_the_script_runs():
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        body = ast.parse(f.read()).body
    guards = [i for i, s in enumerate(body) if isinstance(s, ast.If) and "__name__" in ast.unparse(s.test)]
    assert guards == [len(body) - 1]
