"""The usage examples of the front page: calls that exist, with arguments that they take."""
import ast
import glob
import inspect
import os
import re

import pytest

from gpu_common import lib

dsa = lib()
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def examples():
    text = "".join(open(f).read() for f in sorted(glob.glob(os.path.join(ROOT, "README*"))))
    return re.findall(r"```python\n(.*?)```", text, re.S)


@pytest.mark.parametrize("i", range(len(examples())))
def test_an_example_s_calls_take_what_they_are_given(i):
    code = ast.parse(examples()[i])
    for node in ast.walk(code):
        if not (isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute)
                and isinstance(node.func.value, ast.Name) and node.func.value.id == "dsa"):
            continue
        if any(isinstance(a, ast.Starred) for a in node.args) or any(k.arg is None for k in node.keywords):
            continue
        call = getattr(dsa, node.func.attr)
        inspect.signature(call).bind(*node.args, **{k.arg: k.value for k in node.keywords})


@pytest.mark.parametrize("i", range(len(examples())))
def test_an_example_makes_the_workspaces_that_it_uses(i):
    made = set()
    for line in ast.parse(examples()[i]).body:
        for node in ast.walk(line):
            if isinstance(node, ast.Name) and isinstance(node.ctx, ast.Load) and re.fullmatch(r"w\w*s\d*", node.id):
                assert node.id in made, f"{node.id}, line {node.lineno}"
        made |= {n.id for n in ast.walk(line) if isinstance(n, ast.Name) and isinstance(n.ctx, ast.Store)}
