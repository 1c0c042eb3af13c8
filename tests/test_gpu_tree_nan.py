"""A query that holds a NaN: its (row, head)'s results are NaN, whether one run
or several work it, and nobody else's bits change."""
import pytest

from test_gpu_tree import Problem

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("name,counts,prefix", [("cut", [1], [5000]), ("whole", [2, 3, 1] * 30, [20, 100, 250] * 30),
                                                ("short", [3], [0])])
def test_a_nan_query_stays_a_nan(cache, name, counts, prefix):
    p = Problem(cache, 20, counts, prefix, "chain", seed=26)
    p.run()
    torch.cuda.synchronize()
    o, lse = p.o.clone(), p.lse.clone()
    row, head = p.N - 1, 7
    p.q[row, head, 5] = float("nan")
    p.o.fill_(7.0)
    p.lse.fill_(7.0)
    p.run()
    torch.cuda.synchronize()
    got = int(p.o[row, head].isnan().sum()), int(p.lse[row, head].isnan())
    assert got == (512, 1)
    p.o[row, head], p.lse[row, head] = o[row, head], lse[row, head]
    assert torch.equal(p.o, o) and torch.equal(p.lse, lse)
    assert int(p.err.item()) == 0
