"""The waits that count loads by hand in the adapters' kernels, against the compiled code (see test_mx_waits.py)."""
import os
import re
import subprocess

import pytest

from bit_gemm_nvfp4_amd import build
from test_mx_waits import MANY, least


def compiled(tmp, source):
    out = tmp / (source + ".s")
    cmd = [build.HIPCC, *build.FLAGS, "-S", "--offload-device-only", os.path.join(build.CSRC, source), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return out.read_text().splitlines()


def functions(lines, kernel):
    found, name = {}, None
    for ln in lines:
        start = re.match(r"^(_Z\w*" + kernel + r"\w+):", ln)
        if start:
            name = start.group(1)
            found[name] = []
        elif name and ".Lfunc_end" in ln:
            name = None
        elif name:
            found[name].append(ln)
    return found


@pytest.fixture(scope="module")
def gemm(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("mx_adapter_waits"), "mx_gemm.hip")


def test_the_form_for_few_rows_with_adapters(gemm):
    staged = {n: f for n, f in functions(gemm, "k_adapter_skinny").items() if any("; rows staged" in ln for ln in f)}
    assert len(staged) == 18  # one, two and three row tiles, 4, 8 and 16 rows, two types of C
    for name, lines in staged.items():
        tiles = int(re.search(r"k_adapter_skinnyILi(\d)E", name).group(1))
        waits = least(lines)
        assert sorted({n for n, _ in waits}) == [0, 5 * tiles], name
        assert all(have >= n for n, have in waits), (name, waits)
        assert sum(n > 0 and have < MANY for n, have in waits) >= 3, name


def test_no_kernel_of_the_adapters_or_groups_keeps_registers_in_memory(tmp_path, gemm):
    texts = ["\n".join(gemm)] + ["\n".join(compiled(tmp_path, s)) for s in ("mx_adapters.hip", "mx_grouped.hip", "mx_route.hip")]
    seen = 0
    for text in texts:
        meta = text[text.index(".amdgpu_metadata"):]
        for block in meta.split("- .agpr_count")[1:]:
            name = re.search(r"\.name:\s+(\S+)", block).group(1)
            if re.search(r"k_adapter_(tile|down|sums)|k_mx_(grouped|route|count|place|combine)", name):
                seen += 1
                assert re.search(r"\.private_segment_fixed_size:\s+(\d+)", block).group(1) == "0", name
    assert seen >= 30 + 4 + 1 + 45 + 8
