"""mla_decode_tree over an e4m3 cache where row scales are far apart, against
plain 64-bit attention: rows that a mask hides, visible rows of little weight
and large scale, and scales that spread over orders of magnitude."""
import numpy as np
import pytest

import latent_attention_decode_absorbed_b200 as mla
from test_gpu_tree import Problem, _dev
from tree_ref import SCALE, attend, pack_mask

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def weight_bound(y, window=8.0):
    """Most that a weight can be off, relative to itself.  y [H, L]: log2 of weight times row scale, -inf where not
    seen.  A tile of 256 rows is carried as x = 16 * 2^(y - reference), the reference at most `window` above the
    tile's largest y, so x >= 2^(4 - window) * 2^(y - largest); x is hi + lo, hi the nearest e4m3 value (half a step:
    2^-4 of x's binade, 2^-10 below 2^-6) and lo the nearest e5m2 value to x - hi (half a step of its binade again
    2^-4 below): 2^-8 of x, below 2^-6 at most 2^-14 or an eighth of x, and 2^-17 (or x) at e5m2's last step."""
    H, L = y.shape
    pad = -L % 256
    t = torch.nn.functional.pad(y, (0, pad), value=-float("inf")).view(H, -1, 256)
    top = t.amax(2, keepdim=True)
    x = torch.exp2(t - torch.where(top.isinf(), torch.zeros_like(top), top) + 4.0 - window)
    small = torch.maximum(torch.minimum(torch.full_like(x, 2.0 ** -14), x / 8), torch.minimum(x, torch.full_like(x, 2.0 ** -17)))
    rel = torch.where(x >= 2.0 ** -6, torch.full_like(x, 2.0 ** -8), small / x.clamp(min=2.0 ** -60))
    return rel.view(H, -1)[:, :L]


def close(q, rows, scales, seen, o, lse, what):
    """o [H, 512] and lse [H] of one drafted token against the formula in 64 bits.  rows [L, 576]: the cached values,
    scales [L]: their row scales, seen [L]."""
    ref, rl, a, _ = attend(q, rows, seen)
    x = rows[seen]
    # scores: 576 fp32 additions, each at most a step off, three more roundings, and the two-term query (components
    # below 2^-9 of the largest are 2^-17 of it off)
    e_s = 580 * 2.0 ** -23 * SCALE * (q.abs() @ x.abs().T).amax(1)
    e_s = e_s + SCALE * 2.0 ** -17 * q.abs().amax(1) * x.abs().sum(1).amax()
    assert bool(((lse - rl).abs() <= e_s + 2.0 ** -20 * (1 + rl.abs())).all()), f"{what}: lse"
    z = SCALE * (q @ rows.T)
    y = torch.where(seen[None], z / np.log(2.0) + scales.log2()[None], torch.full_like(z, -float("inf")))
    p = torch.where(seen[None], (z - rl[:, None]).exp(), torch.zeros_like(z))
    tol = (p * weight_bound(y)) @ rows[:, :512].abs() + (2 * e_s[:, None] + 2.0 ** -18) * a + 2.0 ** -22 * ref.abs()
    worst = float(((o - ref).abs() / (tol + 1e-30)).max())
    assert worst <= 1, f"{what}: {worst:.2f}x the bound"
    err = float((o - ref).norm() / ref.norm())
    assert err <= 1e-2, f"{what}: {err:.2e} of the norm"


def check_nodes(p, vals, scale, nodes):
    """The given (sequence, node) pairs of a Problem whose cached values are vals."""
    torch.cuda.synchronize()
    for b, i in nodes:
        n, L = p.counts[b], p.lens[b]
        at = torch.arange(L, device="cuda")
        slots = p.table[b, at // 64].long() * 64 + at % 64
        seen = torch.ones(L, dtype=torch.bool, device="cuda")
        seen[L - n:] = _dev(p.seen[b][i])
        r = int(p.start[b]) + i
        close(p.q[r].double(), vals[slots], scale.view(-1)[slots].double(), seen, p.o[r].double(), p.lse[r].double(),
              f"sequence {b} node {i}")


def values(p):
    codes = mla.unpack_cache_rows(p.pool).view(torch.float8_e4m3fn)
    return codes.double() * p.scale.view(-1).double()[:, None]


@pytest.mark.parametrize("cache,factor", [("bf16", 1.0), ("e4m3", 32.0), ("e4m3", 256.0), ("e4m3", 1e3), ("e4m3", 1e30)])
def test_hidden_drafted_rows_change_nothing(cache, factor):
    """A drafted row that no node sees, and one that only it sees itself, hold the largest finite values: nobody else's
    bits change, and the one that sees itself follows the formula."""
    p = Problem(cache, 64, [7, 5], [300, 30], "tree", seed=21, o_dtype="f32")
    for b, n in enumerate(p.counts):
        s = p.seen[b]
        s[:, 2] = False                      # seen by nobody
        s[:, 3] = False                      # seen by itself only
        s[3, 3] = True
        s[0, 0] = True
        p.mask[int(p.start[b]):int(p.start[b]) + n, 0] = _dev(pack_mask(s, 1))[:, 0]
    p.run()
    torch.cuda.synchronize()
    first, lse = p.o.clone(), p.lse.clone()
    rows = mla.unpack_cache_rows(p.pool).clone()
    alone = []
    for b, n in enumerate(p.counts):
        for k in (2, 3):
            j = p.lens[b] - n + k
            slot = int(p.bt[b, j // 64]) * 64 + j % 64
            if cache == "bf16":
                rows[slot] = 3e4 if k == 2 else rows[slot] * 8
            else:
                if k == 2:
                    rows[slot] = 0x7E        # 448
                p.scale.view(-1)[slot] *= factor if k == 2 else min(factor, 32.0)
        alone.append(int(p.start[b]) + 3)
    p.pool.copy_(mla.pack_cache_rows(rows))
    p.run()
    torch.cuda.synchronize()
    others = [r for r in range(p.N) if r not in alone]
    assert torch.equal(first[others], p.o[others]) and torch.equal(lse[others], p.lse[others])
    assert int(p.err.item()) == 0
    if cache == "e4m3":
        check_nodes(p, values(p), p.scale, [(0, 3), (1, 3), (0, 0), (1, 4)])


@pytest.mark.parametrize("factor", [32.0, 1e3, 1e5])
def test_a_large_row_of_no_weight_takes_nothing_from_the_others(factor):
    p = Problem("e4m3", 32, [3, 2], [900, 150], "chain", seed=22, o_dtype="f32")
    # every query's rope part is 1: a row whose rope codes are -448 has no weight at any of these scales
    p.q[:, :, 512:] = 1.0
    rows = mla.unpack_cache_rows(p.pool).clone()
    for b, at in ((0, 5), (0, 700), (1, 64)):
        slot = int(p.bt[b, at // 64]) * 64 + at % 64
        rows[slot, 512:] = 0xFE              # -448
        p.scale.view(-1)[slot] *= factor
    p.pool.copy_(mla.pack_cache_rows(rows))
    p.run()
    check_nodes(p, values(p), p.scale, [(0, 0), (0, 2), (1, 1)])
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("spread", [1.0, 2.5])
def test_scales_over_orders_of_magnitude(spread):
    p = Problem("e4m3", 128, [4, 2], [1400, 300], "tree", seed=23, q_std=0.02, o_dtype="f32")
    g = torch.Generator(device="cuda")
    g.manual_seed(23)
    p.scale.mul_(torch.exp(spread * torch.randn(p.scale.shape, generator=g, device="cuda")))
    p.run()
    check_nodes(p, values(p), p.scale, [(0, 0), (0, 3), (1, 1)])


def test_zero_rows_and_tiny_scales():
    """Rows of scale zero (an all-zero row) weigh e^0; rows of scale 2^-40 keep their weight in the sum."""
    p = Problem("e4m3", 16, [2, 1], [400, 63], "chain", seed=24, q_std=0.1, o_dtype="f32")
    rows = mla.unpack_cache_rows(p.pool).clone()
    for b, at, sc in ((0, 3, 0.0), (0, 4, 0.0), (0, 399, 2.0 ** -40), (1, 10, 0.0)):
        slot = int(p.bt[b, at // 64]) * 64 + at % 64
        if sc == 0.0:
            rows[slot] = 0
        p.scale.view(-1)[slot] = sc
    p.pool.copy_(mla.pack_cache_rows(rows))
    p.run()
    torch.cuda.synchronize()
    vals = values(p)
    for b, i in ((0, 1), (1, 0)):
        n, L = p.counts[b], p.lens[b]
        at = torch.arange(L, device="cuda")
        slots = p.table[b, at // 64].long() * 64 + at % 64
        seen = torch.ones(L, dtype=torch.bool, device="cuda")
        seen[L - n:] = _dev(p.seen[b][i])
        r = int(p.start[b]) + i
        close(p.q[r].double(), vals[slots], p.scale.view(-1)[slots].double().clamp(min=2.0 ** -48), seen, p.o[r].double(),
              p.lse[r].double(), f"sequence {b} node {i}")


def test_only_zero_rows():
    """A sequence of all-zero rows: o is 0, lse the logarithm of their number."""
    p = Problem("e4m3", 16, [3], [70], "chain", seed=25, o_dtype="f32")
    p.pool.zero_()
    p.scale.zero_()
    p.run()
    torch.cuda.synchronize()
    assert bool((p.o[:3] == 0).all())
    want = torch.log(torch.arange(71, 74, device="cuda", dtype=torch.float64))[:, None]
    assert bool(((p.lse[:3].double() - want).abs() <= 2.0 ** -18).all())
