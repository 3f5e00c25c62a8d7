"""The README's examples use the library as its header allows."""
import ast
import os
import re

import speculative_decoding_verification_masked_gb300 as va

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _blocks():
    with open(README) as f:
        return re.findall(r"```python\n(.*?)```", f.read(), flags=re.S)


def _calls(block):
    for node in ast.walk(ast.parse(block)):
        if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute) and \
                isinstance(node.func.value, ast.Name) and node.func.value.id == "va":
            yield node.func.attr, {k.arg for k in node.keywords}


def test_the_examples_call_what_there_is():
    names = [name for block in _blocks() for name, _ in _calls(block)]
    assert names and all(hasattr(va, n) for n in names)


def test_a_cache_that_is_evicted_shapes_no_distances():
    """Slots of an evicted cache are not positions: a window or slopes over it would
    hide and weigh other tokens than the model does."""
    evicting = [dict(_calls(b)) for b in _blocks() if "verify_evict_kv" in b]
    assert evicting
    for calls in evicting:
        assert not {"window", "slopes"} & calls.get("ScoreMod", set())
