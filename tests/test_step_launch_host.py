"""Decode-step kernels launched ahead of their stream's order, by reading their
source. CPU only."""

import os
import re

import pytest

import linear_attention_state_chunked_gb300 as L

CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")
WAIT = 'asm volatile("griddepcontrol.wait;"'


def kernels_that_wait():
    """(name, body) of every kernel that waits for the launch before it."""
    found = []
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__[^;{]*?(\w+)\(const Plan p\) \{", text):
            body = text[m.end():text.index("\n}", m.end())]
            if WAIT in body:
                found.append((m.group(1), body))
    return found


def test_both_joins_are_found():
    assert [n for n, _ in kernels_that_wait()] == ["join_kernel", "join_row_kernel"]


@pytest.mark.parametrize("name,body", kernels_that_wait(), ids=[n for n, _ in kernels_that_wait()])
def test_no_path_ends_before_the_wait(name, body):
    """What comes next in the stream is ordered behind the early launch alone. A
    grid of which no block waits may end before the launch it belongs to: then
    the next kernel would run beside that one, and could change what it reads or
    get the memory that it still writes."""
    before = body[:body.index(WAIT)]
    assert not re.search(r"\b(return|exit)\b", before), name


def test_a_wait_that_ran_out_leaves_its_items_out():
    """The joins skip an item of which any part is marked. (No wait can be made to
    run out from outside, so this reads the source as well.) A range that gives up
    has two parts at most to answer for: the piece at hand, which is the first
    part where it goes on from the range before, and the second one, of an item
    that goes on past the range."""
    with open(os.path.join(CSRC, "attn_umma.cuh")) as f:
        text = f.read()
    dead = text[text.index("if (s_dead) {"):]
    dead = dead[:dead.index("break;")]
    assert re.search(r"if \(x >= RP \|\| w\.t0 > 0\)\s+p\.part_ml\[2 \* int64_t\(blockIdx\.x\) \* RP \+ x\] = "
                     r"make_float2\(-INFINITY, kLeftOut\)", dead)
    for name, body in kernels_that_wait():
        skip = re.search(r"out \|= ml\S*\.y == kLeftOut;.*?return;", body, re.S)
        assert skip and "p.a.out" not in body[:skip.end()], name
