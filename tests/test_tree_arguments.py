"""Tensors that StepPlan and TreeDecodeStep refuse (no GPU): the kernels read
them by address, so a short or strided one would be read past its end, one of
another type as other numbers."""
import pytest

from latent_attention_decode_absorbed_b200 import StepPlan, TreeDecodeStep
from latent_attention_decode_absorbed_b200 import tree as tree_module

torch = pytest.importorskip("torch")
B, ROWS, H = 3, 12, 4


@pytest.fixture
def made(monkeypatch):
    """A plan and a layer on the CPU, and the names of the library calls that they make."""
    calls = []
    for name in ("mla_step_plan", "mla_cache_append_slots", "mla_absorb_q", "mla_out_uv", "mla_cache_commit"):
        monkeypatch.setattr(tree_module, name, lambda *a, _n=name, **k: calls.append(_n))
    plan = StepPlan(batch=B, num_pages=4, max_pages=2, max_rows=ROWS, device="cpu")
    return plan, TreeDecodeStep(plan, n_heads=H), calls


def _i32(n):
    return torch.zeros(n, dtype=torch.int32)


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


GOOD = {
    "plan": (lambda p, s, x: p.plan(*x), [_i32(B), _i32(ROWS)]),
    "commit": (lambda p, s, x: p.commit([s], *x), [_i32(B), _i32(ROWS)]),
    "append": (lambda p, s, x: s.append(*x), [_bf(ROWS, 576)]),
    "absorb": (lambda p, s, x: s.absorb(*x), [_bf(ROWS, H, 128), _bf(ROWS, H, 64), _bf(H, 128, 512)]),
    "project_out": (lambda p, s, x: s.project_out(*x), [_bf(H, 128, 512)]),
}


@pytest.mark.parametrize("name", sorted(GOOD))
def test_what_fits_is_taken(made, name):
    plan, step, calls = made
    fn, x = GOOD[name]
    fn(plan, step, x)
    fn(plan, step, [torch.cat([t, t]) if t.shape[0] != H else t for t in x])      # more rows than needed
    fn(plan, step, [t.reshape(-1) for t in x])
    fn(plan, step, [t.data_ptr() for t in x] if name != "append" else x)          # addresses
    assert len(calls) == 4


@pytest.mark.parametrize("how", ["short", "dtype", "narrow", "strided"])
@pytest.mark.parametrize("name,which", [(n, i) for n in sorted(GOOD) for i in range(len(GOOD[n][1]))])
def test_what_does_not_fit_is_refused(made, name, which, how):
    plan, step, calls = made
    fn, x = GOOD[name]
    x = list(x)
    t = x[which]
    x[which] = {"short": t[:-1], "dtype": t.to(torch.int64 if t.dtype == torch.int32 else torch.float16),
                "narrow": t[..., :-8].contiguous(),
                "strided": torch.cat([t, t])[::2]}[how]
    with pytest.raises(ValueError):
        fn(plan, step, x)
    assert not calls


def test_another_device_s_tensor_is_refused(made):
    plan, step, calls = made
    plan.cuda = True
    with pytest.raises(ValueError, match="is on cpu"):
        plan.plan(_i32(B))
    assert not calls
