"""The wait of the adapters' first product that counts loads by hand, against the compiled code (see test_mx_waits.py).

k_adapter_down keeps NST - 1 chunks of LOADS loads into LDS in flight.  In front of the barrier that opens a chunk it waits until at
most (NST - 2) LOADS are outstanding, which are the chunks behind if at least as many have been issued behind it: on every
way there the chunk's own loads and those have to be pending."""
import re

import pytest

from test_mx_adapter_waits import compiled, functions
from test_mx_waits import blocks_of


def pending(lines):
    """[(loads that the wait leaves outstanding, fewest loads pending in front of it)] of a function."""
    blocks = blocks_of(lines)

    def walk(body, n):
        waits = []
        body = [ln for ln in body if ln.strip() and not ln.strip().startswith(";")]
        for ln, nxt in zip(body, body[1:] + [""]):
            wait = re.match(r"^\s+s_waitcnt.*vmcnt\((\d+)\)", ln)
            if re.match(r"^\s+buffer_load_dwordx4 .* lds$", ln):
                n += 1
            elif wait and "s_barrier" in nxt and int(wait.group(1)) > 0:
                waits.append((int(wait.group(1)), n))
                n = min(n, int(wait.group(1)))
            elif wait:
                n = min(n, int(wait.group(1)))
        return n, waits
    at, todo = {"entry": 0}, ["entry"]
    while todo:
        b = todo.pop()
        n, _ = walk(blocks[b][0], at[b])
        for nxt in blocks[b][1]:
            if n < at.get(nxt, 1 << 20):
                at[nxt] = n
                todo.append(nxt)
    return [w for b in at for w in walk(blocks[b][0], at[b])[1]]


@pytest.fixture(scope="module")
def down(tmp_path_factory):
    return functions(compiled(tmp_path_factory.mktemp("mx_down_waits"), "mx_adapters.hip"), "k_adapter_down")


def test_each_chunk_has_the_loads_behind_it_that_its_wait_counts(down):
    assert len(down) == 4
    for name, lines in down.items():
        rm, rn, _, nst = map(int, re.search(r"ILi(\d)ELi(\d)ELi(\d)ELi(\d)E", name).groups())
        loads = rm + rn
        waits = pending(lines)
        assert [n for n, _ in waits] == [(nst - 2) * loads], name  # one loop
        assert all(have >= n + loads for n, have in waits), (name, waits)
        # with one load of the loop, or of those in front of it, gone, the count is short
        for gone in [i for i, ln in enumerate(lines) if re.match(r"^\s+buffer_load_dwordx4 .* lds$", ln)]:
            short = pending(lines[:gone] + lines[gone + 1:])
            assert any(have < n + loads for n, have in short), (name, lines[gone])
