"""The row-tile kernels' assembly, as built, keeps what their LDS-direct loads rely on.

The loads are written as instructions, of which the compiler knows nothing, so
what they need is checked on its output (no GPU):
- a load comes five wait states after anything before its block, the rest that
  a memory request needs after a vector instruction wrote a scalar operand;
- m0 has no other use in these kernels;
- a wait that leaves N requests outstanding has at least N requests between it
  and the last LDS-direct load on every way there, so that load is done.
"""
import heapq
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WAIT = re.compile(r"s_waitcnt vmcnt\((\d+)\)$")
REQUEST = re.compile(r"(buffer|global|scratch|flat)_(load|store|atomic)")


def _kernels(text):
    """{kernel: [(instruction, in an inline block)]}; a label is ("name:", False)."""
    kernels, name, block = {}, None, False
    for line in text.splitlines():
        line = line.strip()
        if line.startswith(".amdhsa") or not line:
            continue
        m = re.match(r"(_Z\w*kernel\w*):", line)
        if m:
            name = kernels.setdefault(m.group(1), [])
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name is None:
            continue
        elif line.startswith(";;#ASMSTART"):
            block = True
            name.append(("#start", True))
        elif line.startswith(";;#ASMEND"):
            block = False
            name.append(("#end", True))
        elif re.match(r"\.LBB\w+:", line):
            name.append((line.split(":")[0] + ":", False))
        elif line[0] not in ".;":
            name.append((line.split(";")[0].strip(), block))
    return {k: v for k, v in kernels.items() if any("offen lds" in i for i, _ in v)}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    from bit_quantized_amd import build as B
    out = str(tmp_path_factory.mktemp("asm") / "rows.s")
    r = subprocess.run([B.HIPCC, *B.FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "rows.hip"), "-o", out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        found = _kernels(f.read())
    assert len(found) >= 20  # stream, run and tile kernels
    return found


def test_loads_come_after_the_rest_their_operands_need(kernels):
    for name, code in kernels.items():
        for at, (ins, block) in enumerate(code):
            if "offen lds" not in ins:
                continue
            assert block, name
            states, i = 0, at - 1
            while code[i][0] != "#start":
                m = re.match(r"s_nop (\d+)$", code[i][0])
                states += int(m.group(1)) + 1 if m else 1
                i -= 1
            assert states >= 5, f"{name}: {states} wait states"


def test_m0_has_no_other_use(kernels):
    for name, code in kernels.items():
        for ins, block in code:
            if re.search(r"\bm0\b", ins):
                assert block and ins.startswith(("s_mov_b32 m0,", "s_add_u32 m0, m0,")), f"{name}: {ins}"


def _ways_back(code):
    """For each instruction the ones that may run right before it."""
    label = {ins[:-1]: i for i, (ins, _) in enumerate(code) if ins.endswith(":")}
    back = [[] for _ in code]
    for i, (ins, _) in enumerate(code):
        m = re.match(r"s_c?branch\w* (\.LBB\w+)", ins)
        if m:
            back[label[m.group(1)]].append(i)
        if not ins.startswith(("s_branch", "s_endpgm", "s_setpc")) and i + 1 < len(code):
            back[i + 1].append(i)
    return back


def _requests_since_lds_load(code, back, at, most):
    """The fewest requests between the last LDS-direct load and `at` on any way (at most `most`)."""
    best, queue = {at: 0}, [(0, at)]
    while queue:
        cost, i = heapq.heappop(queue)
        if cost >= most:
            return most
        if cost > best[i]:
            continue
        for p in back[i]:
            ins = code[p][0]
            if "offen lds" in ins:
                return cost
            c = cost + bool(REQUEST.match(ins))
            if c < best.get(p, 1 << 30):
                best[p] = c
                heapq.heappush(queue, (c, p))
    return most


def test_waits_leave_no_lds_load_outstanding(kernels):
    """The waits stand between two empty inline blocks."""
    seen = {}
    for name, code in kernels.items():
        back = _ways_back(code)
        for i, (ins, _) in enumerate(code):
            m = WAIT.match(ins)
            if not m or code[i - 2][0] != "#start" or code[i - 1][0] != "#end" or code[i + 1][0] != "#start":
                continue
            n = int(m.group(1))
            seen[name] = seen.get(name, 0) + 1
            if n:
                got = _requests_since_lds_load(code, back, i, n)
                assert got >= n, f"{name}: {got} requests before a wait that leaves {n}"
    assert set(seen) == set(kernels)  # every kernel has such a wait
