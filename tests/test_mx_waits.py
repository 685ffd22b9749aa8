"""The counted waits of the tile kernels of the grouped MX product, on the
assembly of the built library (no GPU).

Rows come to LDS by DMA, and a wavefront reads rows that others fetched: at
every barrier all of a wavefront's DMAs must have landed.  Its waits count the
loads that may still be on their way (`vmcnt`; loads end in the order they were
issued), so a wait for N covers a DMA exactly where N loads at least are newer
on every path.  The order of loads is the compiler's within what the source
pins down; this test walks all paths of the kernels as they were compiled.
"""
import os
import re
import shutil
import struct
import subprocess

import pytest

import quantized_moe_expert_top_amd as q

NONE_PENDING = 1 << 20  # no DMA since a wait that covered the last one


def objdump():
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    root = os.path.dirname(os.path.dirname(os.path.realpath(hipcc)))
    for d in (root, "/opt/rocm"):
        for sub in ("llvm/bin", "lib/llvm/bin", "bin"):
            p = os.path.join(d, sub, "llvm-objdump")
            if os.path.exists(p):
                return p
    return shutil.which("llvm-objdump")


def code_objects(path):
    """The gfx950 ELF images of a library's offload bundles."""
    data = open(path, "rb").read()
    magic, at = b"__CLANG_OFFLOAD_BUNDLE__", 0
    while (at := data.find(magic, at)) >= 0:
        p = at + len(magic)
        (n,) = struct.unpack_from("<Q", data, p)
        p += 8
        for _ in range(n):
            off, size, name = struct.unpack_from("<QQQ", data, p)
            triple = data[p + 24:p + 24 + name].decode()
            p += 24 + name
            if "gfx950" in triple and size:
                yield data[at + off:at + off + size]
        at += len(magic)


def kernels(text):
    """{name: [(address, mnemonic, operands, branch target or None)]} of a listing."""
    out, name = {}, None
    for line in text.splitlines():
        m = re.match(r"^([0-9a-f]+) <(.+)>:$", line)
        if m:
            name, base = m[2], int(m[1], 16)
            out[name] = []
            continue
        m = re.match(r"^\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if m and name:
            t = re.search(r"<[^>+]*(?:\+0x([0-9a-f]+))?>", m[4])
            target = base + int(t[1] or "0", 16) if t else None
            out[name].append((int(m[3], 16), m[1], m[2], target))
    return out


def uncovered(code):
    """Addresses of barriers that some path reaches with a DMA that no wait covers.  Per instruction the least number
    of loads newer than the last uncovered DMA, over all paths (a store is not counted: it may end out of order)."""
    index = {a: i for i, (a, _, _, _) in enumerate(code)}
    state, todo, bad = {0: NONE_PENDING}, [0], set()
    while todo:
        i = todo.pop()
        newer = state[i]
        a, op, args, target = code[i]
        if op.startswith(("buffer_load", "global_load", "flat_load", "scratch_load")):
            newer = 0 if re.search(r"\blds\b", args) else min(newer + 1, NONE_PENDING)
        elif op == "s_waitcnt":
            m = re.search(r"vmcnt\((\d+)\)", args)
            if m and int(m[1]) <= newer:
                newer = NONE_PENDING
        elif op == "s_barrier" and newer < NONE_PENDING:
            bad.add(a)
        follow = [] if op in ("s_endpgm", "s_branch") else [i + 1]
        if op.startswith(("s_branch", "s_cbranch")):
            follow.append(index[target])
        assert op not in ("s_setpc_b64", "s_swappc_b64"), "calls are not followed"
        for j in follow:
            if j < len(code) and newer < state.get(j, NONE_PENDING + 1):
                state[j] = newer
                todo.append(j)
    return sorted(bad)


def line(i, text, target=None):
    return f"\t{text}  // {4 * i:012X}: 00000000" + (f" <k+0x{4 * target:x}>" if target is not None else "")


def listing(*texts):
    return kernels("0000000000000000 <k>:\n" + "\n".join(line(i, *t) if isinstance(t, tuple) else line(i, t)
                                                       for i, t in enumerate(texts)))["k"]


def test_walk_by_hand():
    """The walk on listings whose answer is plain: a wait that covers, one short of it, and a loop."""
    dma, load, end = "buffer_load_dwordx4 v1, s[0:3], s4 offen lds", "buffer_load_dword v2, v1, s[0:3], s4 offen", "s_endpgm"
    w = "s_waitcnt vmcnt({}) lgkmcnt(0)".format
    assert uncovered(listing(dma, load, load, w(2), "s_barrier", end)) == []
    assert uncovered(listing(load, dma, load, w(2), "s_barrier", end)) == [16]  # a load moved before the DMA
    assert uncovered(listing(dma, "s_barrier", end)) == [4]
    assert uncovered(listing(dma, load, "global_store_dword v[0:1], v2, off", w(2), "s_barrier", end)) == [16]
    # a branch around a load, and the DMA of a loop's last round
    assert uncovered(listing(dma, ("s_cbranch_scc1 1", 3), load, load, w(2), "s_barrier", end)) == [20]
    loop = [dma, load, w(1), "s_barrier", dma, load, ("s_cbranch_scc1 65531", 2), w(0), "s_barrier", end]
    assert uncovered(listing(*loop)) == []
    loop[5] = "v_nop"
    assert uncovered(listing(*loop)) == [12]


def test_tile_kernels_wait_for_their_rows(tmp_path):
    tool = objdump()
    if tool is None:
        pytest.skip("no llvm-objdump")
    assert os.path.exists(q.LIB_PATH), "build the library first"
    checked = 0
    for n, image in enumerate(code_objects(q.LIB_PATH)):
        if b"mx_tile_kernel" not in image:
            continue
        f = tmp_path / f"{n}.elf"
        f.write_bytes(image)
        text = subprocess.run([tool, "-d", str(f)], capture_output=True, text=True, check=True).stdout
        for name, code in kernels(text).items():
            if "mx_tile" in name:
                assert any(re.search(r"\blds\b", c[2]) for c in code), name
                assert uncovered(code) == [], name
                checked += 1
    assert checked == 30, checked  # 6 epilogues: 64 and 128 rows of either format, K split of e2m1 rows
