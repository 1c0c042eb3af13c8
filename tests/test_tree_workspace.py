"""Workspace sizes of mla_decode_tree (no GPU): one for a model's largest step
has to hold every smaller step."""
import pytest

import latent_attention_decode_absorbed_b200 as mla
from latent_attention_decode_absorbed_b200 import build as mla_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    mla_build.build()
    return mla.lib()


@pytest.mark.parametrize("cache", [mla.MLA_F32, mla.MLA_BF16, mla.MLA_E4M3])
def test_more_rows_or_heads_never_need_less(cache):
    size = mla.mla_decode_tree_workspace_bytes
    heads = [1, 2, 15, 16, 17, 31, 32, 33, 48, 64, 65, 100, 127, 128]
    last = [0] * len(heads)
    for rows in list(range(1, 700)) + [1000, 1183, 1184, 1185, 5000, 65535]:
        now = [size(cache, rows, h) for h in heads]
        assert all(a <= b for a, b in zip(now, now[1:])), rows
        assert all(a <= b for a, b in zip(last, now)), rows
        last = now


def test_fp32_holds_every_split():
    """A call of rows x heads leaves ceil(592 / CTAs) partials per (row, head), at most 64, a CTA taking 16 heads."""
    for heads in (1, 5, 16, 17, 33, 128):
        for rows in list(range(1, 700)) + [1000, 5000]:
            splits = min(64, -(-592 // (rows * -(-heads // 16))))
            assert mla.mla_decode_tree_workspace_bytes(mla.MLA_F32, rows, heads) >= rows * heads * splits * 513 * 4
