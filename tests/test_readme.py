"""The Python calls that README.md shows name things that exist and pass
arguments that the functions take, and are those that the GPU tests run (no
GPU)."""
import ast
import inspect
import os

import quantized_moe_expert_top_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_in_the_readme_fit_their_functions():
    blocks = open(os.path.join(ROOT, "README.md")).read().split("```")[1::2]
    checked = 0
    for block in blocks:
        if "q." not in block:
            continue
        for node in ast.walk(ast.parse(block)):
            if isinstance(node, ast.Attribute) and isinstance(node.value, ast.Name) and node.value.id == "q":
                assert hasattr(q, node.attr), node.attr
            if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute) and node.func.value.id == "q":
                inspect.signature(getattr(q, node.func.attr)).bind(*node.args, **{k.arg: k.value for k in node.keywords})
                checked += 1
    assert checked >= 8


def test_gpu_tests_run_the_calls_of_the_readme():
    from tests.test_gpu_mx_edges import README_CALLS
    assert "```\n" + README_CALLS + "```" in open(os.path.join(ROOT, "README.md")).read()
