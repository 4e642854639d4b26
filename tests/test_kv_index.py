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
        '        if (!strcmp(f, "divide")) r = uzkv::divide(a, b);\n'
        '        if (!strcmp(f, "share_of")) r = uzkv::share_of(a, b, c);\n'
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


def test_division_of_any_size(calc):
    r = random.Random(2)
    edge = [1, 2, 3, (1 << 32) - 1, 1 << 32, (1 << 32) + 1, 3 << 32, (1 << 63) - 1]
    calls = [("divide", x, d, 0) for x in edge + [0] for d in edge]
    calls += [("divide", r.getrandbits(r.randint(1, 63)), r.getrandbits(r.randint(1, 63)) | 1, 0) for _ in range(5000)]
    assert calc(calls) == [x // d for _, x, d, _ in calls]


def test_a_position_is_in_the_share_that_holds_it(calc):
    """The join asks which CTA has a tile; the CTAs cut the positions by total * c // shares."""
    r = random.Random(3)
    calls = []
    for bits in (8, 20, 31, 32, 33, 40, 54):  # a total of 2^32 positions has a low word of zero
        for total in [1 << bits] + [r.randint(1, (1 << bits) - 1) for _ in range(150)]:
            shares = min(total, r.choice([1, 7, 148, 152, 160]))
            spots = [0, total - 1, r.randrange(total)] + [total * c // shares + o for c in (1, shares // 2, shares - 1) for o in (-1, 0)]
            calls += [("share_of", at, shares, total) for at in spots if 0 <= at < total]
    for (_, at, shares, total), c in zip(calls, calc(calls)):
        assert total * c // shares <= at < total * (c + 1) // shares


def test_the_join_and_the_split_divide_through_the_helpers():
    """Totals and offsets of the split are 64-bit: no 32-bit division of them remains."""
    join = open(os.path.join(CSRC, "attention.cu")).read()
    split = open(os.path.join(CSRC, "kv_attention.cuh")).read()
    assert "share_of(start" in join and "(uint32_t)total" not in join
    assert "divide(in, width)" in split and "(uint32_t)(at - start)" not in split
