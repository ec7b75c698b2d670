"""Properties of the compiled kernels of the layer norm, dropout and the
vocabulary's loss, from their gfx950 assembly and the compiler's resource
report.  CPU only: the code is cross-compiled here.

* No kernel spills; the loss's 256x256 kernels keep two waves per SIMD with the
  whole 160 KiB of LDS, and their contraction loop one wait for copies, which
  leaves the four youngest under way; the shape for short contractions keeps
  four waves per SIMD and 32 KiB.
* The norm keeps four waves per SIMD or more, which its gradient's grid counts
  on (16 per CU).
* M0 belongs to the direct copies alone, and no packed fp32 instruction is
  emitted (the build disables them)."""

from __future__ import annotations

import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from dense_fp32_tiled_amd import build


@pytest.fixture(scope="module")
def compiled():
    """({source's name: assembly}, resource report of all kernels)."""
    with ThreadPoolExecutor(8) as pool:
        texts = {s.stem: pool.submit(build.device_assembly, s) for s in build.MORE_SOURCES}
        reports = [pool.submit(build.resource_report, s) for s in build.MORE_SOURCES]
        report = {}
        for r in reports:
            report.update(r.result())
        return {k: t.result() for k, t in texts.items()}, report


def big_kernels(names):
    return [n for n in names if "linear_tile_kernel" in n and "LinearShapeILi256ELi256E" in n]


def test_no_kernel_spills(compiled):
    _, report = compiled
    # the norm's shapes, its gradient's, rows that are read again, dropout and the join; the loss's logits of both passes, the
    # gradients' products with what joins their slices, and what stands around them
    assert len(report) >= 3 * 12 + (10 + 10 + 8) + 3 * 3 + 3 * 2 + 1 + 2 * (20 + 5 + 8 + 4) + 4
    assert not {k: v["scratch"] for k, v in report.items() if v.get("scratch", 0) != 0}


def test_tiles_keep_their_occupancy(compiled):
    _, report = compiled
    big = big_kernels(report)
    assert len(big) == 2 * (2 + 2 + 3)
    short = 0
    for name, r in report.items():
        if name in big:
            assert r["occupancy"] == 2 and r["lds"] == 160 * 1024, name
        elif "LinearShapeILi128ELi128ELi64ELi64ELi1ELi4E" in name:
            assert r["occupancy"] >= 4 and r["lds"] == 32 * 1024, name
            short += 1
        elif "linear_tile_kernel" in name:
            assert r["lds"] <= 80 * 1024 and r["occupancy"] >= 2, name
        elif "norm_grad_kernel" in name or "norm_kernel" in name:
            assert r["occupancy"] >= 4, (name, r)
    assert short == 2 * (2 + 2 + 1)


def test_largest_tiles_wait_once_per_contraction_tile(compiled):
    texts, _ = compiled
    seen = 0
    for text in texts.values():
        labels = [(m.start(), m.group(1)) for m in re.finditer(r"^(_Z\w+):", text, re.M)]
        for k, (pos, name) in enumerate(labels):
            if not big_kernels([name]):
                continue
            body = text[pos:labels[k + 1][0] if k + 1 < len(labels) else len(text)]
            loops = [b for b in re.split(r"^\.LBB\d+_\d+:", body, flags=re.M)
                     if len(re.findall(r"^\s+v_mfma_f32_16x16x32", b, re.M)) == 64]
            assert len(loops) == 1, name
            loop = loops[0][:loops[0].index("s_cbranch")]
            assert re.findall(r"s_waitcnt[^\n]*vmcnt\((\d+)\)", loop) == ["4"], name
            seen += 1
    assert seen == 2 * (2 + 2 + 3)


def test_no_packed_fp32_instructions(compiled):
    for text in compiled[0].values():
        assert not re.search(r"v_pk_(?:fma|mul|add)_f32", text)


def test_m0_is_used_only_by_the_direct_copies(compiled):
    uses = 0
    for text in compiled[0].values():
        lines = [l.strip() for l in text.splitlines()]
        code = [l for l in lines if l and not l.startswith((";", ".", "//")) and not l.endswith(":")]
        for i, line in enumerate(code):
            if re.search(r"\bm0\b", line):
                assert re.fullmatch(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)", line), line
                assert code[i + 1] == "s_nop 0", code[i + 1]
                assert re.fullmatch(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], 0 offen lds", code[i + 2]), code[i + 2]
                uses += 1
    assert uses > 100
