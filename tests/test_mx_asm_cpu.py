"""The microscaled tile kernels' assembly, as built, keeps what their LDS-direct
loads rely on (test_rows_asm_cpu.py states the first two for the row tiles):
- a load comes five wait states after anything before its block;
- m0 has no other use;
- the barriers of the main loop leave exactly the loads of the stages behind
  the one that is read next, the second of an iteration also the scales that
  the first let go, and the loop has no other request to memory.
"""
import os
import re
import subprocess

import pytest

import test_rows_asm_cpu as rows

BARRIER = re.compile(r"s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    from bit_quantized_amd import build as B
    out = str(tmp_path_factory.mktemp("asm") / "mx_tile.s")
    r = subprocess.run([B.HIPCC, *B.FLAGS, "--cuda-device-only", "-S", os.path.join(B.CSRC, "mx_tile.hip"), "-o", out],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    with open(out) as f:
        found = rows._kernels(f.read())
    assert len(found) == 32  # two formats, four tiles; whole, in slices, groups, gated groups
    return found


def test_loads_come_after_the_rest_their_operands_need(kernels):
    rows.test_loads_come_after_the_rest_their_operands_need(kernels)


def test_m0_has_no_other_use(kernels):
    rows.test_m0_has_no_other_use(kernels)


def _shape(name):
    """(loads of a stage, loads of scales, buffers) of a kernel, from its template arguments."""
    fmt, wm, wn, fm, fn, kind = map(int, re.search(r"ILi(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d)E", name).groups())
    tall, blocks, waves = 32 * wm * fm, 2 * wn * fn, wm * wn
    row_kib = tall * (128 if fmt else 64) // 1024
    scales = (tall + 16 * blocks) // 64
    room = (160 if waves > 4 else 80) - scales
    third = 160 / 3 - scales
    if kind >= 2 and blocks <= 8 and third >= 3 * (row_kib + blocks):
        room = third
    return (row_kib + blocks) // waves, -(-scales // waves), min(int(room // (row_kib + blocks)), 4)


def _loop(code):
    """The instructions of the innermost loop that holds the products."""
    label = {ins[:-1]: i for i, (ins, _) in enumerate(code) if ins.endswith(":")}
    best = None
    for i, (ins, _) in enumerate(code):
        m = re.match(r"s_c?branch\w* (\.LBB\w+)", ins)
        if m and label[m.group(1)] < i:
            body = [c[0] for c in code[label[m.group(1)]:i]]
            if any("mfma" in c for c in body) and (best is None or len(body) < len(best)):
                best = body
    return best


def test_barriers_leave_the_stages_that_are_not_read_next(kernels):
    for name, code in kernels.items():
        loads, scales, buffers = _shape(name)
        body = _loop(code)
        waits = [i for i, c in enumerate(body) if BARRIER.match(c) and body[i + 1].startswith("s_barrier")]
        assert len(waits) == 2, name
        assert not any(c.startswith(("scratch", "global", "flat")) for c in body), name
        # requests after each barrier, around the loop: stage t + buffers of steps 0 and 1
        span = body[waits[0]:waits[1]], body[waits[1]:] + body[:waits[0]]
        sent = [sum("offen lds" in c for c in s) for s in span]
        assert [sum(bool(rows.REQUEST.match(c)) for c in s) for s in span] == sent, name
        assert sent == [loads + scales, loads], name  # the first brings the scales as well, before the stage
        left = [int(BARRIER.match(body[w]).group(1)) for w in waits]
        # The first leaves whole stages and no scales: those of the iteration
        # before were sent before the oldest of the stages that it leaves.
        assert buffers - 2 <= 2 and left == [(buffers - 2) * loads, (buffers - 2) * loads + scales], name


def test_loads_without_records_have_no_scalar_offset(kernels):
    """The bounds check may subtract the scalar offset from the records: past
    the last stage, where there are none, it must be 0 too."""
    for name, code in kernels.items():
        body = _loop(code)

        def origin(i, reg):
            """The instruction that chose `reg` before instruction i, through shifts and products of it."""
            for back in range(1, len(body)):  # around the loop
                m = re.match(r"(s_\w+) (s\d+), (.*)$", body[i - back])
                if not m or m.group(2) != reg or m.group(1).startswith("s_cmp"):
                    continue
                if not m.group(1).startswith(("s_lshl", "s_mul")):
                    return body[i - back]
                reg = m.group(3).split(",")[0].strip()
            return ""  # set before the loop

        chosen = 0
        for i, c in enumerate(body):
            m = re.match(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], (s\d+) offen lds", c)
            if not m:
                continue
            chosen += bool(re.match(r"s_cselect_b32 s\d+, s\d+, 0$", origin(i, m.group(1))))
        loads, _, _ = _shape(name)
        assert chosen == 2 * loads, name  # (all but the load of scales, which never passes the last super)
