"""What no result shows reliably, read from the gfx950 assembly that hipcc makes of the
experts' products and their gradients: their barriers are bare, so that loads stay in flight
across them, and each wait is the source's own."""
import os
import re
import subprocess

import pytest

from moe_glue_amd import build

SOURCES = ["grouped_linear.hip", "grouped_few.hip", "grouped_grad.hip"]


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    out = {}
    for src in SOURCES:
        path = tmp_path_factory.mktemp("listing") / (src + ".s")
        subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(build.CSRC, src),
                        "-o", str(path)], check=True, capture_output=True)
        out[src] = path.read_text()
    return out


def functions(text):
    """{name: (instructions [(line, op, args)], {label: index of the instruction behind it})}."""
    out, body, labels = {}, None, None
    for number, line in enumerate(text.splitlines(), 1):
        line = line.split(";")[0].strip()
        start = re.match(r"(_Z\w+):$", line)
        label = re.match(r"(\.LBB\w+):$", line)
        if start:
            body, labels = [], {}
            out[start[1]] = (body, labels)
        elif line.startswith(".Lfunc_end"):
            body = None
        elif body is None:
            continue
        elif label:
            labels[label[1]] = len(body)
        elif line and not line.startswith((".", "#")):
            op, _, args = line.partition(" ")
            body.append((number, op, args.strip()))
    return out


def barriers_with_writes_under_way(body, labels):
    """(write, barrier) lines: an LDS write that some path carries to a barrier with no wait
    for it.  Paths by the branches, taken or not."""
    reach = [None] * len(body)      # line of an unfinished write before each instruction, 0: none
    todo, found = [(0, 0)], set()
    while todo:
        i, write = todo.pop()
        while i < len(body):
            if reach[i] is not None and reach[i] >= write:
                break
            reach[i] = write
            number, op, args = body[i]
            if op.startswith("ds_write"):
                write = number
            elif op == "s_waitcnt" and "lgkmcnt(0)" in args:
                write = 0
            elif op == "s_barrier" and write:
                found.add((write, number))
                write = 0
            if op == "s_endpgm":
                break
            if op == "s_branch":
                i = labels[args]
                continue
            if op.startswith("s_cbranch"):
                todo.append((labels[args], write))
            i += 1
    return sorted(found)


def test_the_reader_sees_a_missing_wait():
    text = """_Zk:
	ds_write_b32 v0, v1
	s_cbranch_vccz .LBB0_2
; %bb.1:
	s_waitcnt vmcnt(0) lgkmcnt(0)
.LBB0_2:
	s_barrier
	s_endpgm
.Lfunc_end0:
"""
    ((body, labels),) = functions(text).values()
    assert barriers_with_writes_under_way(body, labels) == [(2, 7)]
    waited = functions(text.replace("s_cbranch_vccz .LBB0_2", "s_waitcnt lgkmcnt(0)"))["_Zk"]
    assert barriers_with_writes_under_way(*waited) == []


@pytest.mark.parametrize("src", SOURCES)
def test_lds_writes_are_done_at_barriers(listings, src):
    """Other waves read behind a barrier what a wave wrote before it: MXFP8 scale bytes that
    are not whole dwords, and the sums of a tile's waves."""
    kernels = functions(listings[src])
    assert sum(op == "s_barrier" for body, _ in kernels.values() for _, op, _ in body) > 0
    for name, (body, labels) in kernels.items():
        found = barriers_with_writes_under_way(body, labels)
        assert not found, f"{src} {name}: (write, barrier) at lines {found}"
