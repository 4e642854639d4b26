"""Index arithmetic of the KV-cache operators at the ends of its range
(csrc/kv_index.cuh), compiled for the host and compared with Python's integers."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lossless_bf16_exponent_gb300", "csrc")


@pytest.fixture(scope="module")
def calc(tmp_path_factory):
    """Runs lines of `name a b c` through the header's functions."""
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("kv_index")
    src = d / "calc.cpp"
    src.write_text(
        '#include "kv_index.cuh"\n#include <inttypes.h>\n#include <stdio.h>\n#include <string.h>\n'
        "int main(void) {\n"
        "    char f[32];\n    uint64_t a, b, c;\n"
        '    while (scanf("%31s %" SCNu64 " %" SCNu64 " %" SCNu64, f, &a, &b, &c) == 4) {\n'
        "        uint64_t r = 0;\n"
        '        if (!strcmp(f, "next_below")) r = uzkv::next_below((uint32_t)a, (uint32_t)b, (uint32_t)c);\n'
        '        printf("%" PRIu64 "\\n", r);\n'
        "    }\n}\n")
    exe = str(d / "calc")
    subprocess.run([cc, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", exe], check=True)

    def run(calls):
        text = "".join(f"{f} {a} {b} {c}\n" for f, a, b, c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [int(v) for v in out.split()]

    return run


def test_steps_end_at_the_total(calc):
    r = random.Random(1)
    calls = [("next_below", 4294967264 - 1, 1245184, 4294967264),  # the largest output of heads of 512 bytes, one row a grid
             ("next_below", 4294967264 - 1245184, 1245184, 4294967264), ("next_below", 4294967264 - 1245185, 1245184, 4294967264),
             ("next_below", 0, 1, 1), ("next_below", 0, 256, 4294967295), ("next_below", 4294967294, 4294967295, 4294967295)]
    for _ in range(2000):
        total = r.randint(1, (1 << 32) - 1)
        calls.append(("next_below", r.randint(max(0, total - (1 << r.randint(1, 32))), total - 1), 1 << r.randint(0, 31), total))
    assert calc(calls) == [min(i + step, total) for _, i, step, total in calls]


def test_packing_steps_through_the_helper():
    """The packing loop takes no unbounded 32-bit step: its indexes go up to what the host accepts, just below 2^32."""
    text = open(os.path.join(CSRC, "evict.cu")).read()
    body = text[text.index("pack_kernel(const"):text.index("launch_select(")]
    assert "next_below(" in body and "i +=" not in body
