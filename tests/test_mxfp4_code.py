"""What the compiler made of the MXFP4 products' kernels: no scratch, and no LDS but what the source counts."""
import re

import pytest

import code_objects as co


@pytest.fixture(scope="module")
def files(tmp_path_factory):
    return co.unbundle(tmp_path_factory.mktemp("code"))


@pytest.fixture(scope="module")
def kernels(files):
    found = {k: v for k, v in co.notes(files).items() if "3moe" in k and "mx_" in k}
    assert len(found) > 30
    return found


def test_no_scratch(kernels):
    """No spilled registers and no arrays in memory: either stands between a step's loads and its products."""
    used = {k: (v["private_segment_fixed_size"], v["vgpr_spill_count"]) for k, v in kernels.items()}
    assert {k: u for k, u in used.items() if any(u)} == {}


def test_lds_is_what_the_tiles_take(kernels):
    """Tiles of TM rows by TN columns in LDS: two steps of rows, two blocks of codes and scales, and nothing that the compiler
    put there by itself (the source checks their sum against the CU's 160 KB)."""
    seen = 0
    for name, fields in kernels.items():
        n = co.template_numbers(name, "mx_kernel")
        if n is None:
            continue
        x4, pair, wm, wn, wgm, wgn = n[:6]
        tm, tn = wm * wgm, wn * wgn
        row_scales = -(-tm * 8 // 256) * 256 if x4 else 0
        weight_scales = -(-(tn // 2 if pair else tn) * 8 // 1024) * 1024 * (2 if pair else 1)
        assert fields["group_segment_fixed_size"] == 2 * tm * 128 + 2 * (tn * 128 + row_scales + weight_scales), name
        seen += 1
    assert seen >= 6


def test_blocks_are_loaded_in_turn(files):
    """The kernels for few rows wait until at most the loads of the later blocks are in flight: that is right while the rows of each
    block go to LDS before a later block's loads, so no more loads into LDS follow one another than a block has."""
    seen = 0
    for name, text in co.code(files, "mx_rows_kernel").items():
        x4, _, fragments, _, waves, depth = co.template_numbers(name, "mx_rows_kernel")
        if depth == 2:  # waits for everything
            continue
        block = 16 * fragments * (128 if x4 else 512) // 1024 // waves  # of a wave
        loads = "".join("L" if m[2] else "r" for m in re.finditer(r"^\s*buffer_load_(dwordx[24])\b.*?( lds)?$", text, re.M))
        assert "r" in loads and max(len(run) for run in loads.split("r")) == block, name
        seen += 1
    assert seen >= 14
