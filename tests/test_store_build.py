"""Build-level check of the stores that go past the caches (no GPU needed): kernels whose lanes write eight
fp32 values, two stores of 16 bytes each, use plain ones. Past the caches, each of the two would leave
every other 16 bytes of a line to the other, and the lines reach memory in halves."""

import os
import re
import subprocess
import tempfile

import pytest

from test_build import BUILD, _tool


def nontemporal_stores(obj):
    """kernel -> number of its stores past the caches."""
    objcopy, bundler, objdump = (_tool(n) for n in ("llvm-objcopy", "clang-offload-bundler",
                                                    "llvm-objdump"))
    if not (os.path.exists(obj) and objcopy and bundler and objdump):
        pytest.skip("kernels not built here, or the ROCm LLVM tools are missing")
    with tempfile.TemporaryDirectory() as tmp:
        fat, dev = os.path.join(tmp, "fatbin"), os.path.join(tmp, "dev.o")
        subprocess.run([objcopy, f"--dump-section=.hip_fatbin={fat}", obj, os.path.join(tmp, "x")],
                       check=True, capture_output=True)
        subprocess.run([bundler, "--unbundle", "--type=o", f"--input={fat}",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--output={dev}"],
                       check=True, capture_output=True)
        text = subprocess.run([objdump, "-d", "--mcpu=gfx950", dev], check=True, capture_output=True,
                              text=True).stdout
    counts, cur = {}, None
    for line in text.splitlines():
        m = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if m:
            cur = m.group(1)
            counts.setdefault(cur, 0)
        elif cur and re.search(r"global_store\S*\s.*\bnt\b", line):
            counts[cur] += 1
    return counts


@pytest.mark.parametrize("source,kernels", [
    ("ssd_conv", "k_conv"), ("ssd_group_norm", "k_gn_(apply|tokens|few|whole)")])
def test_no_half_lines_past_the_caches(source, kernels):
    counts = nontemporal_stores(os.path.join(BUILD, source + ".o"))
    ours = {k: n for k, n in counts.items() if re.search(kernels, k) and not k.endswith(".kd")}
    fp32 = {k: n for k, n in ours.items() if re.search(kernels + "If", k)}
    assert fp32 and any(n for k, n in ours.items() if k not in fp32), sorted(ours)
    assert not any(fp32.values()), fp32
