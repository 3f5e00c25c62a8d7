"""TMEM loads are asynchronous: their registers may be read only after the wait.
Only a wait that names the registers keeps the compiler from moving what reads
them before it, so every load's array has to be handed to one."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_masked_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
LOAD = re.compile(r"\btmem_ld(?:8|16|32)\(")
WAIT = re.compile(r"\btmem_ld_wait\w*\(([^()]*)\)")


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _last_argument(s, start):
    """The last argument of the call whose parenthesis opens before `start`."""
    depth, last, i = 1, start, start
    while depth:
        if s[i] in "([":
            depth += 1
        elif s[i] in ")]":
            depth -= 1
        elif s[i] == "," and depth == 1:
            last = i + 1
        i += 1
    return s[last:i - 1].strip()


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_every_tmem_load_is_tied_to_its_wait(path):
    s = _code(path)
    assert path.endswith("va_tcgen05.cuh") or "tcgen05.wait::ld" not in s
    for m in LOAD.finditer(s):
        if s[:m.start()].rstrip().endswith("void"):  # the definition
            continue
        array = _last_argument(s, m.end()).split("[")[0]
        # the nearest following waits of the same few statements: one of them names the array
        waits = [w.group(1) for w in WAIT.finditer(s, m.end(), m.end() + 700)]
        named = {a.split("[")[0].strip() for w in waits for a in w.split(",")}
        assert array in named, f"{os.path.basename(path)}: load of {array} at {s.count(chr(10), 0, m.start()) + 1} has no tied wait"


def test_a_wait_names_registers():
    for path in FILES:
        s = _code(path)
        for m in WAIT.finditer(s):
            if s[:m.start()].rstrip().endswith("void"):
                continue
            assert m.group(1).strip(), f"{os.path.basename(path)}: a wait without registers"
