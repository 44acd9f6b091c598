"""What no result shows reliably, read from the gfx950 assembly that hipcc makes of the
experts' products and their gradients: their barriers are bare, so that loads stay in flight
across them, and each wait is the source's own; and their loads to LDS are assembly, whose
operands the compiler keeps no wait states for."""
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


WAIT_STATES = 5  # between a vector instruction that writes a scalar register and a load that reads it


def scalars(args):
    """Numbers of the scalar registers in an operand list."""
    found = {int(n) for n in re.findall(r"\bs(\d+)\b", args)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", args):
        found.update(range(int(a), int(b) + 1))
    return found


def loads_too_early(body, labels):
    """(write, load) lines: a scalar register that a vector instruction writes and a load to
    LDS reads fewer than WAIT_STATES wait states later on some path."""
    after = [[] for _ in body]
    for i, (_, op, args) in enumerate(body):
        if op == "s_branch" or op.startswith("s_cbranch"):
            after[i].append(labels[args])
        if op not in ("s_branch", "s_endpgm") and i + 1 < len(body):
            after[i].append(i + 1)
    found = set()
    for i, (number, op, args) in enumerate(body):
        if not op.startswith("v_"):
            continue
        out = args.split(",")
        written = scalars(out[0]) | (scalars(out[1]) if "_co_" in op or "div_scale" in op else set())
        todo = [(j, 0, written) for j in after[i]] if written else []
        while todo:
            j, states, left = todo.pop()
            if j >= len(body) or states >= WAIT_STATES:
                continue
            line, op2, args2 = body[j]
            if op2.startswith("buffer_load") and "lds" in args2.split() and scalars(args2) & left:
                found.add((number, line))
            if op2.startswith("s_") and not op2.startswith(("s_waitcnt", "s_cmp", "s_cbranch", "s_nop", "s_bitcmp")):
                left = left - scalars(args2.split(",")[0])     # the scalar unit's own later value
            wait = int(args2, 0) + 1 if op2 == "s_nop" else 1
            todo += [(n, states + wait, left) for n in after[j]] if left else []
    return sorted(found)


def test_the_reader_sees_a_load_too_early():
    text = """_Zk:
	v_readfirstlane_b32 s6, v1
	s_cbranch_vccz .LBB0_2
; %bb.1:
	s_nop 4
.LBB0_2:
	s_mov_b32 m0, s2
	s_nop 0
	buffer_load_dwordx4 v1, s[4:7], s9 offen lds
	s_endpgm
.Lfunc_end0:
"""
    assert loads_too_early(*functions(text)["_Zk"]) == [(2, 9)]
    for other in (text.replace("s6, v1", "s3, v1"), text.replace("s_nop 0", "s_nop 2"),
                  text.replace("s_cbranch_vccz .LBB0_2", "s_add_i32 s6, s6, 1")):
        assert loads_too_early(*functions(other)["_Zk"]) == []


@pytest.mark.parametrize("src", ["grouped_linear.hip", "grouped_grad.hip"])
def test_scalar_operands_of_loads_are_settled(listings, src):
    loads = 0
    for name, (body, labels) in functions(listings[src]).items():
        loads += sum(op.startswith("buffer_load") and "lds" in args.split() for _, op, args in body)
        found = loads_too_early(body, labels)
        assert not found, f"{src} {name}: (write, load) at lines {found}"
        # M0 is written for each load and read by nothing that has an operand of that name
        assert not [n for n, op, args in body if "m0" in args and not (op == "s_mov_b32" and args.startswith("m0,"))]
    assert loads > 0


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
