"""Limits of the MX layer's calls that are checked on the host, without a GPU."""
import ctypes

import pytest

import quantized_moe_expert_top_amd as q

BAD_SHAPE, BAD_FORMAT = 2, 3


@pytest.fixture(scope="module")
def lib():
    return q.lib()


def layer_call(lib, T, k=1, E=1, H=128, I=128, **kw):
    """moe_mx_layer on addresses that no check refuses, but for what `kw` changes."""
    descs = []
    for N, K in ((2 * I, H), (H, I)):
        d = q.MxDesc()
        d.abi_version, d.layout, d.E, d.N, d.K = q.MOE_ABI_VERSION, q.MOE_LAYOUT_TILED, E, N, K
        d.codes, d.scales = 0x10000, 0x20000
        descs.append(d)
    f = dict(abi_version=q.MOE_ABI_VERSION, T=T, k=k, x_dtype=q.MOE_DTYPE_BF16, x_fmt=1, h_fmt=1, y_dtype=q.MOE_DTYPE_F16,
             kernel=0, score=0, n_group=1, topk_group=1, group_top=1, renormalize=1, scale=1.0,
             gate_up=ctypes.pointer(descs[0]), down=ctypes.pointer(descs[1]))
    for i, n in enumerate(("x", "logits", "topk_ids", "topk_w", "expert_counts", "seg_offsets", "sorted_pair", "pair_pos",
                           "workspace", "x_codes", "x_scales", "h_codes", "h_scales", "y", "out")):
        f[n] = 0x100000 * (i + 1)
    f["workspace_bytes"] = 1 << 40
    f.update(kw)
    layer = q.MxLayer()
    for n, v in f.items():
        setattr(layer, n, v)
    return lib.moe_mx_layer(ctypes.byref(layer), None)


def test_layer_refuses_more_tokens_than_its_combine_takes(lib):
    """Every launch of a layer must be possible before the first one runs; y_dtype is checked behind T."""
    for T in (1 << 24, (1 << 24) + 1, (1 << 25) - 1):
        assert layer_call(lib, T, y_dtype=9) == BAD_SHAPE
        assert b"2^24" in lib.moe_last_error_detail()
    assert layer_call(lib, (1 << 24) - 1, y_dtype=9) == BAD_FORMAT


def test_layer_workspace_next_to_the_largest_pair_count(lib):
    """No size comes from a pair count that overflows when it is rounded up to whole chunks."""
    size = lib.moe_mx_layer_workspace_size
    for T, k in ((2099201, 1023), (33038209, 65), (8259545, 260)):
        assert 2 ** 31 - 2048 < T * k < 2 ** 31 and size(T, k, 1024) == 0
    nb = -(-2097000 * 1023 // 2048)  # chunks of pairs, a flag and 1025 counters each
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    assert size(2097000, 1023, 1024) == 256 + up(4 * nb) + up(4 * 1025 * nb)
