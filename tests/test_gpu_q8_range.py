"""mla_decode_fwd_q8 where softmax weights or row scales are far apart within a
split, against plain 64-bit attention with the two-term query: a strong early
row before a long thin tail, and a visible row of large scale and no weight."""
import numpy as np
import pytest

import latent_attention_decode_absorbed_b200 as mla
from test_gpu_tree_range import Sink
from test_gpu_tree_scales import close
from tree_ref import SCALE

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _decode(q, pool, scale, pages, table, length, heads, split):
    """The partials of one query row, and the query that its codes stand for."""
    q8 = torch.empty((1, 2, heads, 576), dtype=torch.uint8, device="cuda")
    qs = torch.empty((1, heads), device="cuda")
    mla.mla_split_q_e4m3(q, 1, heads, q8, qs)
    n = -(-table.shape[1] * 64 // split)
    o = torch.full((1, heads, n, 512), float("nan"), device="cuda")
    lse = torch.full((1, heads, n), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_decode_fwd_q8(q8, qs, pool, scale, pages, table, table.shape[1], 64,
                          torch.tensor([length], dtype=torch.int32, device="cuda"), 1, 1, heads, n, split, SCALE, o, lse, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    terms = q8[0].view(torch.float8_e4m3fn).double()
    return o[0], lse[0], (terms[0] + terms[1]) * qs[0].double()[:, None]


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("mass", [0.3, 0.5, 0.9])
@pytest.mark.parametrize("length", [1024, 4096, 32768])
def test_one_split_keeps_a_thin_tail(length, mass, same):
    s = Sink(length, mass, 1, 128, seed=41, same=same)
    o, lse, q = _decode(s.q, s.pool, s.scale, s.pages, s.table, length, 128, s.pages * 64)
    rows = s.codes.double() * s.row_scale.double()[:, None]
    seen = torch.ones(length, dtype=torch.bool, device="cuda")
    close(q, rows, s.row_scale.double(), seen, o[:, 0].double(), lse[:, 0].double(), f"{length} rows")


@pytest.mark.parametrize("factor", [32.0, 1e3, 1e5])
def test_a_large_row_of_no_weight_takes_nothing_from_the_others(factor):
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    length, heads, pages = 700, 96, 11
    x = torch.randn((pages * 64, 576), generator=g, device="cuda")
    amax = x.abs().amax(1)
    codes = (x * (448.0 / amax)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = amax / 448.0
    for at in (5, 300):                     # rope codes -448 against a query whose rope part is 1
        codes[at, 512:] = 0xFE
        scale[at] *= factor
    q = (torch.randn((1, heads, 576), generator=g, device="cuda") * 0.6).to(torch.bfloat16)
    q[..., 512:] = 1.0
    table = torch.tensor(np.arange(pages, dtype=np.int32)[None], device="cuda")
    o, lse, qd = _decode(q, mla.pack_cache_rows(codes), scale.view(pages, 64), pages, table, length, heads, pages * 64)
    rows = codes[:length].view(torch.float8_e4m3fn).double() * scale[:length].double()[:, None]
    seen = torch.ones(length, dtype=torch.bool, device="cuda")
    close(qd, rows, scale[:length].double(), seen, o[:, 0].double(), lse[:, 0].double(), "large row")
