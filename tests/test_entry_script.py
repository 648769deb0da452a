"""``python __graft_entry__.py smoke`` finds every function of the file: what runs as a script is its last statement."""
import ast
import os


def test_the_script_part_comes_last():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "__graft_entry__.py")
    with open(path, encoding="utf-8") as f:
        body = ast.parse(f.read()).body
    scripts = [i for i, s in enumerate(body) if isinstance(s, ast.If) and "__name__" in ast.unparse(s.test)]
    assert scripts == [len(body) - 1]
