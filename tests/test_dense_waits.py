"""The tile kernels of the 16-bit products as they were compiled (no GPU):
their DMAs are waited for before every barrier, and their stores are of the
form whose data the next instruction may overwrite."""
import os
import re
import subprocess

import pytest

import quantized_moe_expert_top_amd as q
from tests.test_mx_waits import code_objects, kernels, listing, objdump, uncovered


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    tool = objdump()
    if tool is None:
        pytest.skip("no llvm-objdump")
    assert os.path.exists(q.LIB_PATH), "build the library first"
    out = {}
    for n, image in enumerate(code_objects(q.LIB_PATH)):
        if b"deep_kernel" in image and b"GemmK" in image:
            f = tmp_path_factory.mktemp("co") / f"{n}.elf"
            f.write_bytes(image)
            text = subprocess.run([tool, "-d", str(f)], capture_output=True, text=True, check=True).stdout
            out.update(kernels(text))
    return {name: code for name, code in out.items() if "kernel" in name}


def waits_before_barriers(code):
    """The vmcnt that was waited for last before each barrier, with no load between (None: none)."""
    out, last = [], None
    for _, op, args, _ in code:
        if op == "s_waitcnt" and (m := re.search(r"vmcnt\((\d+)\)", args)):
            last = int(m[1])
        elif op.startswith(("buffer_load", "global_load", "flat_load", "scratch_load", "s_branch", "s_cbranch")):
            last = None
        elif op == "s_barrier":
            out.append(last)
            last = None
    return out


def wide_stores(code):
    """Stores of more than 8 bytes through a descriptor whose scalar offset is a register."""
    return [args for _, op, args, _ in code
            if re.match(r"buffer_store_(dwordx[34]|b96|b128)", op) and not re.search(r"s\[\d+:\d+\], 0\b", args)]


def test_readings_by_hand():
    dma, end = "buffer_load_dwordx4 v1, s[0:3], s4 offen lds", "s_endpgm"
    w = "s_waitcnt vmcnt({}) lgkmcnt(0)".format
    assert waits_before_barriers(listing(dma, w(8), "s_barrier", dma, "s_barrier", w(0), dma, "s_barrier", end)) == [8, None, None]
    assert wide_stores(listing("buffer_store_dwordx4 v[0:3], v4, s[0:3], 0 offen nt", end)) == []
    assert len(wide_stores(listing("buffer_store_dwordx4 v[0:3], v4, s[0:3], s7 offen", end))) == 1
    assert wide_stores(listing("buffer_store_dword v0, v4, s[0:3], s7 offen", end)) == []


def test_tiles_wait_for_their_dmas(compiled):
    """Two stages: nothing is on its way at a barrier.  Three: the DMAs of one step, 8 (128 x 128) or 12 (128 x 256)."""
    two = {n: c for n, c in compiled.items() if "11tile_kernel" in n}
    three = {n: c for n, c in compiled.items() if "11deep_kernel" in n}
    assert len(two) == 32 and len(three) == 12, (len(two), len(three))
    for name, code in two.items():
        assert any(re.search(r"\blds\b", c[2]) for c in code), name
        assert uncovered(code) == [], name
    for name, code in three.items():
        waits = waits_before_barriers(code)
        assert waits and all(v is not None and v <= 12 for v in waits), (name, waits)
        assert {8, 12} <= set(waits), (name, waits)


def test_stores_have_no_scalar_offset(compiled):
    """gfx950 may store what the instruction behind such a store writes to its data registers, and the compiler sees no
    hazard in it (seen in these kernels before their stores added the row's offset to the lanes' own)."""
    for name, code in compiled.items():
        assert wide_stores(code) == [], name
