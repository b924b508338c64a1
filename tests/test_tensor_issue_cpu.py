"""What the fifth-generation tensor core's kernels rest on and no run can show: a commit covers the products of the thread that makes
it and of no other, so products and commits are named by the one thread that elect() names, which is no thread of a known number."""

import pathlib
import re

import pytest

import sparse_slot_memory_gb300 as sdm

CSRC = pathlib.Path(sdm.__file__).parent / "csrc"
NAMED = re.compile(r"tensor::(mma|commit)\(")


def headers(text, at):
    """The statements that open the blocks around a place."""
    stack, start = [], 0
    for i, c in enumerate(text[:at]):
        if c == "{":
            stack.append(text[start:i])
        elif c == "}":
            stack.pop()
        if c in "{};":
            start = i + 1
    return stack


def issues():
    for path in sorted(CSRC.glob("sdm_*.cu")):
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", path.read_text(), flags=re.S)
        for m in NAMED.finditer(text):
            yield path.name, text.count("\n", 0, m.start()) + 1, headers(text, m.start())


def test_there_are_products_and_commits():
    assert len(list(issues())) > 20


@pytest.mark.parametrize("name", sorted({n for n, _, _ in issues()}))
def test_products_and_commits_are_the_elected_thread_s(name):
    others = [line for n, line, around in issues() if n == name and not any("tensor::elect()" in h for h in around)]
    assert not others, f"{name}: products or commits of another thread than the elected one, about line {others}"
