"""Host-side checks of the drafted-step operators (no GPU): every refusal, and
the workspace sizes.  The pointers are never dereferenced."""
import math

import pytest

import latent_attention_decode_absorbed_b200 as mla
from latent_attention_decode_absorbed_b200 import build as mla_build

FAKE = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    mla_build.build()
    return mla.lib()


def _refused(fn, kw, status):
    with pytest.raises(mla.MlaError) as e:
        fn(**kw)
    assert e.value.status == status
    assert mla.lib().mla_last_error_message().decode().startswith(fn.__name__ + ":")


PLAN = dict(seq_lens=FAKE, new_counts=FAKE + 256, parents=FAKE, batch=2, max_rows=8, mask_words=1, held_in=FAKE + 512,
            held_out=FAKE + 512, free_pages=FAKE, free_count_in=FAKE, free_count_out=FAKE, block_table=FAKE,
            max_pages_per_seq=4, page_size=64, num_pages=8, row_start=FAKE + 768, kv_lens=FAKE + 1024, seq_ids=None,
            positions=FAKE, slots=FAKE, tree_mask=FAKE, err_word=None, stream=0)
INV, UNS = mla.MLA_ERR_INVALID_ARG, mla.MLA_ERR_UNSUPPORTED


@pytest.mark.parametrize("over,status", [
    (dict(page_size=32), UNS), (dict(batch=0), INV), (dict(max_rows=-1), INV), (dict(num_pages=0), INV),
    (dict(max_pages_per_seq=0), INV), (dict(mask_words=0), INV), (dict(mask_words=-1, tree_mask=None), INV),
    (dict(num_pages=1 << 25), UNS), (dict(max_pages_per_seq=1 << 25), UNS), (dict(batch=1 << 30), UNS),
    (dict(seq_lens=None), INV), (dict(held_out=None), INV), (dict(free_pages=None), INV), (dict(slots=None), INV),
    (dict(positions=None), INV), (dict(kv_lens=FAKE), INV), (dict(row_start=FAKE + 256), INV),
    (dict(held_out=FAKE), INV),
])
def test_step_plan_refusals(over, status):
    _refused(mla.mla_step_plan, {**PLAN, **over}, status)


APPEND = dict(kv_a=FAKE, kv_dtype=mla.MLA_BF16, n_new=4, slots=FAKE, positions=FAKE, norm_gain=None, eps=1e-6,
              rope_cos=FAKE, rope_sin=FAKE, rope_max_pos=64, cache=FAKE, cache_scale=FAKE, cache_dtype=mla.MLA_E4M3,
              num_pages=4, err_word=None, stream=0)


@pytest.mark.parametrize("over,status", [
    (dict(n_new=-1), INV), (dict(kv_dtype=mla.MLA_E4M3), UNS), (dict(cache_dtype=7), UNS), (dict(num_pages=0), INV),
    (dict(rope_max_pos=0), INV), (dict(num_pages=1 << 25), UNS), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(slots=None), INV), (dict(cache=None), INV), (dict(cache_scale=None), INV), (dict(kv_a=FAKE + 8), INV),
    (dict(norm_gain=FAKE + 4), INV),
])
def test_append_slots_refusals(over, status):
    _refused(mla.mla_cache_append_slots, {**APPEND, **over}, status)


TREE = dict(q_abs=FAKE, q_dtype=mla.MLA_BF16, cache=FAKE, cache_scale=None, cache_dtype=mla.MLA_BF16, num_pages=4,
            block_table=FAKE, max_pages_per_seq=4, page_size=64, kv_lens=FAKE, row_start=FAKE, batch=1, max_rows=8,
            n_heads=128, tree_mask=FAKE, mask_words=1, softmax_scale=1 / math.sqrt(192), workspace=FAKE, o_lat=FAKE,
            o_dtype=mla.MLA_BF16, lse_out=None, err_word=None, stream=0)


@pytest.mark.parametrize("over,status", [
    (dict(page_size=16), UNS), (dict(batch=0), INV), (dict(max_rows=-1), INV), (dict(n_heads=0), INV),
    (dict(n_heads=129), INV), (dict(mask_words=0), INV), (dict(softmax_scale=0.0), INV),
    (dict(softmax_scale=math.inf), INV), (dict(q_dtype=mla.MLA_F32), UNS), (dict(cache_dtype=mla.MLA_F32), UNS),
    (dict(o_dtype=mla.MLA_E4M3), UNS), (dict(max_pages_per_seq=1 << 25), INV), (dict(max_rows=1 << 22), UNS),
    (dict(q_dtype=mla.MLA_F32, cache_dtype=mla.MLA_F32, max_rows=65536, n_heads=1), UNS), (dict(q_abs=None), INV),
    (dict(num_pages=3728271), UNS),
    (dict(workspace=None), INV), (dict(o_lat=None), INV), (dict(cache_dtype=mla.MLA_E4M3), INV),
    (dict(cache=FAKE + 64), INV), (dict(workspace=FAKE + 8), INV), (dict(tree_mask=FAKE + 4), INV),
    (dict(q_abs=FAKE + 2), INV),
])
def test_decode_tree_refusals(over, status):
    _refused(mla.mla_decode_tree, {**TREE, **over}, status)


COMMIT = dict(kv_lens=FAKE, row_start=FAKE + 256, batch=2, max_rows=8, accept_counts=FAKE + 512, accept_nodes=FAKE,
              block_table=FAKE, max_pages_per_seq=4, page_size=64, cache=FAKE, cache_scale=None,
              cache_dtype=mla.MLA_BF16, num_pages=4, seq_lens_out=FAKE + 768, err_word=None, stream=0)


@pytest.mark.parametrize("over,status", [
    (dict(page_size=128), UNS), (dict(batch=0), INV), (dict(max_rows=-1), INV), (dict(num_pages=0), INV),
    (dict(cache_dtype=9), UNS), (dict(max_pages_per_seq=1 << 25), INV), (dict(accept_nodes=None), INV),
    (dict(cache=None), INV), (dict(seq_lens_out=FAKE), INV), (dict(seq_lens_out=FAKE + 512), INV),
    (dict(cache_dtype=mla.MLA_E4M3), INV), (dict(cache=FAKE + 8), INV),
])
def test_commit_refusals(over, status):
    _refused(mla.mla_cache_commit, {**COMMIT, **over}, status)


def test_zero_rows_enqueue_nothing():
    mla.mla_cache_append_slots(**{**APPEND, "n_new": 0, "kv_a": None, "slots": None, "cache": None})
    mla.mla_decode_tree(**{**TREE, "max_rows": 0, "q_abs": None, "workspace": None})


def test_workspace_bytes():
    size = mla.mla_decode_tree_workspace_bytes
    # bf16: two partials of 128 rows (512 numbers and a log-normaliser) for each of 96 pairs, whatever the rows
    assert size(mla.MLA_BF16, 1, 1) == size(mla.MLA_BF16, 1000, 128)
    assert 2 * 96 * 128 * 513 * 4 <= size(mla.MLA_BF16, 1, 1) < 2 * 96 * 128 * 513 * 4 + 8192
    # e4m3: also the two-term query and its scales
    more = size(mla.MLA_E4M3, 1000, 128) - size(mla.MLA_BF16, 1000, 128)
    assert 128000 * (2 * 576 + 4) <= more < 128000 * (2 * 576 + 4) + 1024
    assert size(mla.MLA_F32, 10, 16) >= 160 * 16 * 513 * 4
    assert size(mla.MLA_BF16, 0, 16) == 0 and size(mla.MLA_BF16, 4, 0) == 0 and size(5, 4, 4) == 0
