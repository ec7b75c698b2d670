"""Properties of the compiled kernels of the products with an epilogue and the
token sort, from their gfx950 assembly and the compiler's resource report.
CPU only: the code is cross-compiled here.

* No kernel spills, and the 256x256 kernels keep two waves per SIMD with the
  whole 160 KiB of LDS.
* Their K loop is one block of 64 MFMAs with one wait for copies, which leaves
  the four youngest under way (a wait that the compiler adds for loads or
  stores of the epilogue would wait for every copy).
* M0 belongs to the direct copies alone, and no packed fp32 instruction is
  emitted (the build disables them)."""

from __future__ import annotations

import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from dense_fp32_tiled_amd import build


@pytest.fixture(scope="module")
def compiled():
    """(assembly of every source, resource report of all kernels)."""
    with ThreadPoolExecutor(6) as pool:
        texts = [pool.submit(build.device_assembly, s) for s in build.LINEAR_SOURCES]
        reports = [pool.submit(build.resource_report, s) for s in build.LINEAR_SOURCES]
        report = {}
        for r in reports:
            report.update(r.result())
        return [t.result() for t in texts], report


def big_kernels(names):
    return [n for n in names if "linear_tile_kernel" in n and "LinearShapeILi256ELi256E" in n]


def test_no_kernel_spills(compiled):
    _, report = compiled
    assert len(report) >= 2 * 3 * 7 + 10
    assert not {k: v["scratch"] for k, v in report.items() if v.get("scratch", 0) != 0}


def test_largest_tiles_keep_their_occupancy(compiled):
    _, report = compiled
    big = big_kernels(report)
    assert len(big) == 2 * 3  # two types, three layouts of the operands
    for name in big:
        assert report[name]["occupancy"] == 2 and report[name]["lds"] == 160 * 1024, name
    for name, r in report.items():
        if "linear_tile_kernel" in name and name not in big:
            assert r["lds"] <= 80 * 1024 and r["occupancy"] >= 2, name


def test_largest_tiles_wait_once_per_contraction_tile(compiled):
    texts, _ = compiled
    seen = 0
    for text in texts:
        labels = [(m.start(), m.group(1)) for m in re.finditer(r"^(_Z\w+):", text, re.M)]
        for k, (pos, name) in enumerate(labels):
            if not big_kernels([name]):
                continue
            body = text[pos:labels[k + 1][0] if k + 1 < len(labels) else len(text)]
            loops = [b for b in re.split(r"^\.LBB\d+_\d+:", body, flags=re.M)
                     if len(re.findall(r"^\s+v_mfma_f32_16x16x32", b, re.M)) == 64]
            assert len(loops) == 1, name
            # up to the branch back: what follows in the same block belongs to the epilogue
            loop = loops[0][:loops[0].index("s_cbranch")]
            waits = re.findall(r"s_waitcnt[^\n]*vmcnt\((\d+)\)", loop)
            assert waits == ["4"], (name, waits)
            seen += 1
    assert seen == 2 * 3


def test_no_packed_fp32_instructions(compiled):
    for text in compiled[0]:
        assert not re.search(r"v_pk_(?:fma|mul|add)_f32", text)


def test_m0_is_used_only_by_the_direct_copies(compiled):
    """The copies write M0 without saving it, which is safe only while no compiler-generated code keeps a value in
    it."""
    uses = 0
    for text in compiled[0]:
        lines = [l.strip() for l in text.splitlines()]
        code = [l for l in lines if l and not l.startswith((";", ".", "//")) and not l.endswith(":")]
        for i, line in enumerate(code):
            if re.search(r"\bm0\b", line):
                assert re.fullmatch(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)", line), line
                assert code[i + 1] == "s_nop 0", code[i + 1]
                assert re.fullmatch(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], 0 offen lds", code[i + 2]), code[i + 2]
                uses += 1
    assert uses > 100
