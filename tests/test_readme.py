"""The README's usage block: what is turned to its positions once is not turned
again, and its calls are the binding's."""
import ast
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def calls():
    """(names assigned, function, names passed) of the block's calls, in order."""
    with open(os.path.join(ROOT, "README.md")) as f:
        block = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "sv.verify(" in b)
    for node in ast.parse(block).body:
        call = node.value if isinstance(node, (ast.Assign, ast.Expr)) else None
        if isinstance(call, ast.Call) and isinstance(call.func, ast.Attribute):
            targets = [n.id for t in getattr(node, "targets", []) for n in ast.walk(t) if isinstance(n, ast.Name)]
            yield targets, call.func.attr, [n.id for a in call.args for n in ast.walk(a) if isinstance(n, ast.Name)]


def test_nothing_is_turned_twice():
    turned, seen = set(), []
    for targets, name, args in calls():
        if name in ("rope", "rope_kv_write"):
            assert not turned & set(args), (name, args)
            turned |= set(targets)
            seen.append(name)
        else:
            turned -= set(targets)
    assert seen == ["rope", "rope_kv_write"]


def test_its_calls_exist():
    import rejection_sampling_verify_03_amd as sv
    names = [name for _, name, _ in calls()]
    assert len(names) > 10 and all(callable(getattr(sv, n)) for n in names)
