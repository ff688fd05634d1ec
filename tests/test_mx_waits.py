"""The waits of the form for few rows that count loads by hand, against the compiled code.

Rows of A pass through LDS by loads that the compiler does not connect with the reads of them, so the kernel waits until
at most N loads are outstanding, N being the loads that it issues behind them.  Were fewer compiled there (one dropped, or
moved ahead), the wait would end too early.  The marks in the assembly show where rows have been staged and where they
are taken as arrived: every way through the code from one to the other has to hold N loads at least.
"""
import os
import re
import subprocess

import pytest

from bit_gemm_nvfp4_amd import build

MANY = 1 << 20
LOAD = re.compile(r"^\s+(global_load|buffer_load|flat_load|scratch_load)")
JUMP = re.compile(r"^\s+s_(c?branch\w*)\s+(\S+)")


def blocks_of(lines):
    """{label: (instructions, successors)} of a function's lines."""
    out, name, body = {}, "entry", []

    def close(nexts):
        out[name] = (body, nexts)
    for ln in lines:
        label = re.match(r"^(\.L\w+):", ln)
        jump = JUMP.match(ln)
        if label:
            close([label.group(1)])
            name, body = label.group(1), []
        elif jump:
            follow = f"{name}+{len(out)}"
            close([jump.group(2)] + ([] if jump.group(1) == "branch" else [follow]))
            name, body = follow, []
        elif "s_endpgm" in ln:
            close([])
            name, body = f"{name}+{len(out)}", []
        else:
            body.append(ln)
    close([])
    return out


def walk(body, n):
    """Loads since the last rows were staged, behind a block that starts with n; the waits on the way."""
    waits = []
    for ln in body:
        if "; rows staged" in ln:
            n = 0
        elif "; rows arrived" in ln:
            waits.append((int(re.search(r"arrived, (\d+)", ln).group(1)), n))
        elif LOAD.match(ln):
            n += 1
    return n, waits


def least(lines):
    """[(loads the wait counts on, fewest loads behind the staged rows)] of a function."""
    blocks = blocks_of(lines)
    at = {b: MANY * 2 for b in blocks}
    todo = ["entry"]
    at["entry"] = MANY
    while todo:
        b = todo.pop()
        n, _ = walk(blocks[b][0], at[b])
        for nxt in blocks[b][1]:
            if n < at[nxt]:
                at[nxt] = n
                todo.append(nxt)
    return [w for b in blocks if at[b] < MANY * 2 for w in walk(blocks[b][0], at[b])[1]]


@pytest.fixture(scope="module")
def functions(tmp_path_factory):
    out = tmp_path_factory.mktemp("mx_waits") / "mx_gemm.s"
    cmd = [build.HIPCC, *build.FLAGS, "-S", "--offload-device-only", os.path.join(build.CSRC, "mx_gemm.hip"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found, name = {}, None
    for ln in out.read_text().splitlines():
        start = re.match(r"^(_Z\w*k_mx_skinny\w+):", ln)
        if start:
            name = start.group(1)
            found[name] = []
        elif name and ".Lfunc_end" in ln:
            name = None
        elif name:
            found[name].append(ln)
    return found


def test_every_way_to_a_wait_holds_the_loads_it_counts(functions):
    staged = {n: f for n, f in functions.items() if any("; rows staged" in ln for ln in f)}
    assert len(staged) == 18  # one, two and three row tiles, 4, 8 and 16 rows, two types of C
    for name, lines in staged.items():
        tiles = int(re.search(r"k_mx_skinnyILi(\d)E", name).group(1))
        waits = least(lines)
        assert sorted({n for n, _ in waits}) == [0, 5 * tiles], name
        assert all(have >= n for n, have in waits), (name, waits)
        assert sum(n > 0 and have < MANY for n, have in waits) >= 3, name  # both steps of the loop, and the last group


CODE = """
	buffer_load_dwordx4 v1, s[0:3], 0 offen lds
	; rows staged
	global_load_dwordx4 v[2:5], v[6:7], off
	s_cbranch_scc1 .LBB0_2
	global_load_dwordx4 v[2:5], v[6:7], off
.LBB0_1:
	; rows arrived, 2 loads behind
	buffer_load_dwordx4 v1, s[0:3], 0 offen lds
	; rows staged
	global_load_dwordx4 v[2:5], v[6:7], off
	buffer_load_dwordx4 v[2:5], v1, s[0:3], 0 offen
	s_cbranch_vccnz .LBB0_1
	s_endpgm
.LBB0_2:
	; rows arrived, 2 loads behind
	s_branch .LBB0_1
"""


def test_the_count_finds_the_way_with_the_fewest_loads():
    # the way over the branch has one load only, and reaches the loop with it; the loop's own way has two
    assert sorted(least(CODE.splitlines())) == [(2, 1), (2, 1)]
    assert sorted(least(CODE.replace("s_cbranch_scc1 .LBB0_2", "s_nop 0").splitlines())) == [(2, 2)]
