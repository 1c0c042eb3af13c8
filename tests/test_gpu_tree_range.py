"""Attention over an e4m3 cache where one early row holds much of the mass and
the rest is spread thin over a long context, the rows sharing a common
component, against plain 64-bit attention."""
import math

import pytest

import latent_attention_decode_absorbed_b200 as mla
from test_gpu_tree_scales import close
from tree_ref import SCALE

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Sink:
    """One sequence of `length` cached rows.  Latents are a common vector plus noise, the first row's the common
    vector's negative; queries are orthogonal to the common vector, scores of the other rows have standard deviation
    1, and the first row's rope part lifts its score to `mass` of the softmax.  same=True: the other rows are alike."""

    def __init__(self, length, mass, tokens, heads, seed, same=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.H, self.T, self.L = heads, tokens, length
        common = rand(512)
        x = torch.zeros((length, 576), device="cuda")
        x[:, :512] = common + (rand(1, 512) if same else rand(length, 512))
        x[0, :512] = -common
        q = rand(tokens, heads, 576) * (math.sqrt(192.0) / math.sqrt(512.0))
        q[..., :512] -= (q[..., :512] @ common / common.square().sum())[..., None] * common
        q[..., 512:] = 1.0
        self.q = q.to(torch.bfloat16)
        # ln of the others' sum: ln L + 1/2 for scores of variance 1
        x[0, 512:] = (math.log(length) + 0.5 + math.log(mass / (1 - mass))) / (64 * SCALE)
        self.pages = -(-length // 64)
        full = torch.zeros((self.pages * 64, 576), device="cuda")
        full[:length] = x
        amax = full.abs().amax(1)
        codes = torch.where(amax[:, None] > 0, full * (448.0 / amax)[:, None], torch.zeros_like(full))
        codes = codes.clamp(-448, 448).to(torch.float8_e4m3fn)
        perm = torch.randperm(self.pages, generator=g, device="cuda")
        self.scale = torch.empty((self.pages, 64), device="cuda")
        self.scale[perm] = (amax / 448.0).view(-1, 64)
        self.pool = torch.empty((self.pages, 9, 64, 64), dtype=torch.uint8, device="cuda")
        self.pool[perm] = mla.pack_cache_rows(codes.view(torch.uint8))
        self.table = perm.to(torch.int32).view(1, -1).contiguous()
        self.codes, self.row_scale = codes[:length], (amax / 448.0)[:length]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(self, row, visible, o, lse):
        rows = self.codes[:visible].double() * self.row_scale[:visible].double()[:, None]
        seen = torch.ones(visible, dtype=torch.bool, device="cuda")
        close(self.q[row].double(), rows, self.row_scale[:visible].double(), seen, o.double(), lse.double(), f"row {row}")


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("mass", [0.3, 0.5, 0.9])
@pytest.mark.parametrize("length", [4096, 32768, 131072])
def test_tree_attention_keeps_a_thin_tail(length, mass, same):
    """80 drafted tokens of 128 heads: more row tiles than CTA pairs, so that a row tile is worked in one run."""
    s = Sink(length, mass, 80, 128, seed=31, same=same)
    o = torch.empty((80, 128, 512), device="cuda")
    lse = torch.empty((80, 128), device="cuda")
    ws = torch.empty(mla.mla_decode_tree_workspace_bytes(mla.MLA_E4M3, 80, 128), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 80], dtype=torch.int32, device="cuda")
    mla.mla_decode_tree(s.q, mla.MLA_BF16, s.pool, s.scale, mla.MLA_E4M3, s.pages, s.table, s.pages, 64, lens, start, 1, 80,
                        128, None, 0, SCALE, ws, o, mla.MLA_F32, lse, s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0
    for i in (0, 40, 79):
        s.check(i, length - 80 + i + 1, o[i], lse[i])
