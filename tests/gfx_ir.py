"""The device code of a source as LLVM IR, and its accesses to LDS on every way through a function."""
import os
import re
import subprocess

from bit_gemm_nvfp4_amd import build

SYNC = re.compile(r"\bfence\b|llvm\.amdgcn\.s\.barrier")
OPS = {"load": "L", "store": "S", "atomicrmw": "X", "cmpxchg": "X"}


def compiled(tmp, source):
    """Lines of the IR of a source of the library."""
    out = os.path.join(str(tmp), source + ".ll")
    cmd = [build.HIPCC, *build.FLAGS, "-S", "-emit-llvm", "--offload-device-only", os.path.join(build.CSRC, source), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    with open(out) as f:
        return f.read().splitlines()


def functions(lines):
    """{mangled name: lines of its body}"""
    found, name = {}, None
    for ln in lines:
        start = re.match(r"^define .*@(\w+)\(", ln)
        if start:
            name = start.group(1)
            found[name] = []
        elif ln.startswith("}"):
            name = None
        elif name:
            found[name].append(ln)
    return found


def blocks_of(lines):
    """{label: (instructions, successors)}; the first block is the entry."""
    out, name = {"entry": ([], [])}, "entry"
    for ln in lines:
        label = re.match(r"^([\w.]+):", ln)
        if label:
            name = label.group(1)
            out[name] = ([], [])
        elif ln.strip():
            out[name][0].append(ln)
            if re.match(r"^\s+(br|switch)\b|^\s+\]|^\s+i\d+ \S+, label", ln):
                out[name][1].extend(re.findall(r"label %([\w.]+)", ln))
    return out


class Lds:
    """A function's accesses to LDS: (kind, type, byte offset of the array in LDS or None, block, index)."""

    def __init__(self, lines):
        self.blocks = blocks_of(lines)
        self.base = {}
        for body, _ in self.blocks.values():
            for ln in body:
                g = re.match(r"^\s+(%[\w.]+) = getelementptr .*?, ptr addrspace\(3\) (.*)$", ln)
                if g:
                    self.base[g.group(1)] = g.group(2)

    def offset(self, operand):
        """Constant offset that the address starts from, found back through the instructions that form it."""
        for _ in range(100):
            name = re.match(r"(%[\w.]+)", operand)
            if name and name.group(1) in self.base:
                operand = self.base[name.group(1)]
                continue
            const = re.match(r"getelementptr [\w ]*\(i8, ptr addrspace\(3\) @\w+, i32 (\d+)\)", operand)
            return int(const.group(1)) if const else 0 if operand.startswith("@") else None

    def steps(self, body):
        """The accesses and the waits ("sync") of a block, in order."""
        for ln in body:
            if SYNC.search(ln):
                yield "sync", None, None
                continue
            g = re.match(r"^\s+(?:%[\w.]+ = )?(?:tail )?(load|store|atomicrmw|cmpxchg)\b(.*)$", ln)
            if g and "addrspace(3)" in g.group(2):
                rest = g.group(2)
                at = rest.index("ptr addrspace(3) ") + len("ptr addrspace(3) ")
                kind = re.match(r"\s*(?:atomic |volatile |add |or )*(<[^>]*>|[\w.]+)", rest).group(1)
                yield OPS[g.group(1)], kind, self.offset(rest[at:])

    def unordered(self, first, then, same_block):
        """[(access, access)]: those that `first` picks and, on some way from there without a wait, those that `then` picks.
        same_block: pairs within one block count too."""
        found = []
        for start, (body, _) in self.blocks.items():
            open_ = set()
            for n, (kind, ty, off) in enumerate(self.steps(body)):
                if kind == "sync":
                    open_.clear()
                    continue
                if same_block:
                    found += [(a, (kind, ty, off, start, n)) for a in open_ if then(kind, ty, off)]
                if first(kind, ty, off):
                    open_.add((kind, ty, off, start, n))
            if not open_:
                continue
            seen, todo = set(), list(self.blocks[start][1])
            while todo:
                b = todo.pop()
                if b in seen:
                    continue
                seen.add(b)
                for n, (kind, ty, off) in enumerate(self.steps(self.blocks[b][0])):
                    if kind == "sync":
                        break
                    if then(kind, ty, off) and (same_block or b != start):
                        found += [(a, (kind, ty, off, b, n)) for a in open_]
                else:
                    todo += self.blocks[b][1]
        return found
