"""The pipelined chunk loops of the built library: when a stage is read, the loads that fill it have been waited for.  The
kernels count vector memory operations (a wave's complete in order), so the counts hold only if the compiled loop issues a
chunk's loads ahead of its stores; here the counts of the machine code itself are checked, loop by loop (CPU)."""
import os
import re
import shutil
import subprocess

import pytest

from tests.test_exec_masks import LIB, code_objects

KERNEL = re.compile(r"linattn_chunk_kernelILi(\d)ELi(\d+)ELi(\d)ELb([01])")


def parse(text):
    """{kernel: [(address, opcode, arguments, branch target or None)]}"""
    out, code = {}, None
    for line in text.splitlines():
        m = re.match(r"([0-9a-f]+) <(\w+)>:", line)
        if m:
            code, start = out.setdefault(m.group(2), []), int(m.group(1), 16)
            continue
        m = re.match(r"\s+([a-z]\w+)\s*(.*?)\s*// ([0-9A-F]+):(.*)", line)
        if m and code is not None:
            t = re.search(r"\+0x([0-9a-f]+)>", m.group(4)) if "branch" in m.group(1) else None
            code.append((int(m.group(3), 16), m.group(1), m.group(2), start + int(t.group(1), 16) if t else None))
    return out


def graph(code):
    """(successors, predecessors) of the instructions by place."""
    place = {c[0]: i for i, c in enumerate(code)}
    succ = [[] for _ in code]
    for i, (_, op, _, target) in enumerate(code):
        if op not in ("s_branch", "s_endpgm") and i + 1 < len(code):
            succ[i].append(i + 1)
        if target in place:
            succ[i].append(place[target])
    pred = [[] for _ in code]
    for i, t in enumerate(succ):
        for j in t:
            pred[j].append(i)
    return succ, pred


def reach(start, edges):
    seen, todo = {start}, [start]
    while todo:
        for j in edges[todo.pop()]:
            if j not in seen:
                seen.add(j)
                todo.append(j)
    return seen


def loops(code):
    """The loops with at least two barriers and loads to LDS, as (code, places): every instruction from which a barrier is
    reached that reaches it again (blocks that the compiler moved out of line among them)."""
    succ, pred = graph(code)
    found, seen = [], set()
    for i, c in enumerate(code):
        if c[1] == "s_barrier" and i not in seen:
            body = reach(i, succ) & reach(i, pred)
            seen |= body
            barriers = sum(code[j][1] == "s_barrier" for j in body)
            if barriers >= 2 and any(code[j][1].startswith("buffer_load") and "lds" in code[j][2] for j in body):
                found.append((code, body))
    return found


def loads_not_waited_for(loop):
    """Loads to LDS that may still be on their way when their stage is read: the loop has a barrier for each stage, and the
    last of those that follow a load opens the turn that reads it.  On the way there, by the path with the fewest vector
    memory operations, there has to be a wait that allows no more of them than have been issued since."""
    code, places = loop
    succ, _ = graph(code)
    at = {c[0]: i for i, c in enumerate(code)}
    stages = sum(code[i][1] == "s_barrier" for i in places)

    def follow(i, left_out):
        """(next place, whether a store has just been left out).  A store of fp32 and one of the dtype stand as the two arms of
        a branch, each behind a jump of its own: of two stores in a row not both are left out."""
        pc, op, _, target = code[i]
        nxt = []
        for j in succ[i]:
            if j not in places:
                continue
            over = target in at and j == at[target] and target > pc and any(
                k in places and code[k][1].startswith("buffer_store") for k in range(i, j))
            if not (over and left_out):
                nxt.append((j, over or (left_out and not op.startswith("buffer_store"))))
        return nxt

    bad = []
    for start in sorted(places):
        pc, op, args, _ = code[start]
        if not (op.startswith("buffer_load") and "lds" in args):
            continue
        fewest, todo = {}, [(j, s, 0, 0) for j, s in follow(start, False)]   # place, .., barriers passed, operations since
        while todo:
            i, left_out, barriers, behind = todo.pop()
            if fewest.get((i, left_out, barriers), behind + 1) <= behind:
                continue
            fewest[i, left_out, barriers] = behind
            _, op, args, _ = code[i]
            if op == "s_waitcnt" and "vmcnt" in args and int(re.search(r"vmcnt\((\d+)\)", args).group(1)) <= behind:
                continue                                        # done by here
            if op == "s_barrier":
                barriers += 1
                if barriers == stages - 1:
                    bad.append(hex(pc))
                    break
            behind += op.startswith(("buffer_", "global_", "scratch_", "flat_"))
            todo += [(j, s, barriers, behind) for j, s in follow(i, left_out)]
    return bad


def test_the_check_sees_a_load_behind_a_store():
    line = "\t%s // %012X: 00000000"
    def body(ops):                                              # noqa: E306
        lines = [line % (o, 4 * i) for i, o in enumerate(ops)]
        lines.append(line % ("s_cbranch_vccnz 1", 4 * len(ops)) + " <k+0x0>")
        return loops(parse("0000000000000000 <k>:\n" + "\n".join(lines))["k"])[0]
    load, store = "buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "buffer_store_dwordx4 v[0:3], v4, s[0:3], 0 offen"
    turn = ["s_waitcnt vmcnt(2) lgkmcnt(0)", "s_barrier", load, load, store, store]
    assert loads_not_waited_for(body(turn * 2)) == []
    late = ["s_waitcnt vmcnt(2) lgkmcnt(0)", "s_barrier", load, store, load, store]
    assert loads_not_waited_for(body(turn + late)) != []
    three = ["s_waitcnt vmcnt(6) lgkmcnt(0)", "s_barrier", load, load, store, store]     # two chunks' stores and a chunk's loads
    assert loads_not_waited_for(body(three * 3)) == []
    assert loads_not_waited_for(body(three * 2 + [three[0], "s_barrier", store, load, load, store])) != []


def test_chunk_loops_wait_for_the_stage_they_read(tmp_path):
    tool = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
    if not os.path.exists(LIB) or not os.path.exists(tool):
        pytest.skip("no built library, or no llvm-objdump")
    checked, bad = 0, []
    for i, elf in enumerate(code_objects(LIB)):
        if b"linattn_chunk_kernel" not in elf:
            continue
        path = tmp_path / f"{i}.elf"
        path.write_bytes(elf)
        r = subprocess.run([tool, "-d", str(path)], stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        assert r.returncode == 0, r.stderr[-500:]
        for name, code in parse(r.stdout).items():
            if KERNEL.search(name):
                inner = loops(code)
                assert len(inner) == 1, (name, len(inner))
                checked += 1
                if loads_not_waited_for(inner[0]):
                    bad.append(KERNEL.search(name).groups())
    assert checked >= 60
    assert not bad, bad
