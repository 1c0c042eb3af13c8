"""mla_cache_commit with impossible lengths and offsets: flagged, nothing moved."""
import numpy as np
import pytest

import latent_attention_decode_absorbed_b200 as mla
from test_gpu_tree import _dev, make_pool

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


# (kv_lens, row_start, count) of one sequence of a call of 8 rows, and its length afterwards (the prefix, 0 where there is none)
@pytest.mark.parametrize("kv,start,count,left", [
    (LOW, [0, 8], 2, 0), (LOW + 7, [0, 8], 2, 0), (-1, [0, 8], 2, 0), (3, [0, 8], 2, 0), (129, [0, 8], 2, 121),
    (HIGH, [0, 8], 2, HIGH - 8), (108, [LOW, 8], 2, 0), (108, [8, 0], 2, 0), (108, [0, HIGH], 2, 0), (108, [0, 9], 2, 0),
    (108, [LOW, HIGH], 2, 0), (108, [0, 8], HIGH, 100), (108, [0, 8], LOW, 100)])
def test_impossible_numbers_move_nothing(kv, start, count, left):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    pool, _, _ = make_pool(gen, 4, "bf16")
    before = pool.clone()
    out = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_commit(_dev(np.array([kv], np.int32)), _dev(np.array(start, np.int32)), 1, 8,
                         _dev(np.array([count], np.int32)), _dev(np.array([3, 5] + [0] * 6, np.int32)),
                         _dev(np.array([[2, 0]], np.int32)), 2, 64, pool, None, mla.MLA_BF16, 4, out, err)
    torch.cuda.synchronize()
    assert int(err.item()) == mla.MLA_DEVERR_POSITION
    assert torch.equal(pool, before)
    assert int(out.item()) == left
