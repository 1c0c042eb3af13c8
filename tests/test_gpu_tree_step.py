"""Drafted decode steps as a serving loop runs them: prompts admitted, trees
drafted, paths committed, sequences finished and replaced, on two layers, eager
and as one captured graph; against plain 64-bit attention over the rows that a
plain append of the accepted tokens stores."""
import numpy as np
import pytest

import latent_attention_decode_absorbed_b200 as mla
from latent_attention_decode_absorbed_b200 import StepPlan, TreeDecodeStep
from tree_ref import SCALE, ancestors, attend, random_parents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
H, B, ROWS, NODES = 16, 5, 160, 20


class Model:
    """Two layers, their weights, and what a plain loop knows of each sequence."""

    def __init__(self, cache, seed):
        self.g = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.cache = cache
        self.dt = torch.float32 if cache == "f32" else torch.bfloat16
        self.plan = StepPlan(batch=B, num_pages=60, max_pages=12, max_rows=ROWS, max_nodes=NODES)
        self.layers = [TreeDecodeStep(self.plan, n_heads=H, dtype="f32" if cache == "f32" else "bf16",
                                      cache_dtype=cache) for _ in range(2)]
        self.w = [(self.rand(H, 128, 512, std=512 ** -0.5), self.rand(H, 128, 512, std=512 ** -0.5))
                  for _ in self.layers]
        self.tokens = [[] for _ in range(B)]      # per sequence: (layer 0's raw row, layer 1's raw row)

    def rand(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.gen, device="cuda") * std).to(self.dt)

    def inputs(self):
        """One step's inputs for both layers: kv_a, q_nope, q_pe."""
        return [(self.rand(ROWS, 576), self.rand(ROWS, H, 128), self.rand(ROWS, H, 64)) for _ in self.layers]

    def stored(self, layer, rows, positions):
        """The rows that mla_cache_append stores for raw rows at positions, in float64."""
        st = self.layers[layer]
        n = len(rows)
        pages = -(-n // 64)
        pool = torch.zeros((pages, 9, 64, 64), dtype=st.cache.dtype, device="cuda")
        scale = torch.zeros((pages, 64), device="cuda")
        code = {torch.float32: mla.MLA_F32, torch.bfloat16: mla.MLA_BF16}[self.dt]
        # one page table entry per position's page: every row in a table of its own sequence
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        width = int(pos.max().item()) // 64 + 1
        slot = torch.arange(n, dtype=torch.int32, device="cuda")
        mla.mla_cache_append_slots(torch.stack(rows), code, n, slot, pos, None, st.eps, st.rope_cos, st.rope_sin,
                                   st.max_pos, pool, scale if self.cache == "e4m3" else None, st.cache_dtype, pages)
        assert width <= 12
        vals = mla.unpack_cache_rows(pool)[:n]
        if self.cache == "e4m3":
            return vals.view(torch.float8_e4m3fn).double() * scale.view(-1)[:n, None].double()
        return vals.double()

    def check_rows(self):
        """The caches hold the accepted tokens' rows, bit for bit, in order."""
        table = self.plan.block_table.cpu().numpy()
        lens = self.plan.seq_lens.tolist()
        for b in range(B):
            assert lens[b] == len(self.tokens[b])
            if not lens[b]:
                continue
            slots = [int(table[b, j // 64]) * 64 + j % 64 for j in range(lens[b])]
            for k, st in enumerate(self.layers):
                got = mla.unpack_cache_rows(st.cache)[slots]
                if self.cache == "e4m3":
                    got = got.view(torch.float8_e4m3fn).double() * st.cache_scale.view(-1)[slots][:, None].double()
                want = self.stored(k, [t[k] for t in self.tokens[b]], list(range(lens[b])))
                assert torch.equal(got.double(), want), f"sequence {b}, layer {k}"

    def check_out(self, ins, counts, seen):
        """Every new row's attention against plain attention over prefix and seen drafted rows."""
        start = np.concatenate([[0], np.cumsum(counts)])
        for k, st in enumerate(self.layers):
            kv, qn, qp = ins[k]
            w_uk, w_uv = (x.double() for x in self.w[k])
            for b in range(B):
                n, old = counts[b], len(self.tokens[b])
                if n == 0:
                    continue
                depth = [int(seen[b][i].sum()) - 1 for i in range(n)]
                rows = self.stored(k, [t[k] for t in self.tokens[b]] + [kv[start[b] + i] for i in range(n)],
                                   list(range(old)) + [old + d for d in depth])
                for i in sorted({0, n // 2, n - 1}):
                    r = int(start[b]) + i
                    q = torch.cat([torch.einsum("hkc,hk->hc", w_uk, qn[r].double()), qp[r].double()], 1)
                    vis = torch.ones(old + n, dtype=torch.bool, device="cuda")
                    vis[old:] = torch.as_tensor(seen[b][i]).cuda()
                    o, _, a, _ = attend(q, rows, vis)
                    want = torch.einsum("hic,hc->hi", w_uv, o)
                    # bf16: q_abs is rounded (2^-8 of each component, scores off by up to that times sum |q k|),
                    # then the weights, o_lat and out (2^-8 each, of sum |w| sum p |c|)
                    big = torch.einsum("hic,hc->hi", w_uv.abs(), a)
                    if self.cache == "f32":
                        tol = 1e-4 * big + 1e-6
                    else:
                        ds = SCALE * 2.0 ** -8 * (q.abs() @ rows.abs().T).amax(1)
                        tol = (3 * 2.0 ** -8 + 2 * ds[:, None]) * big + 1e-6
                    err = (st.out[r].double() - want).abs()
                    assert bool((err <= tol).all()), f"seq {b} node {i} layer {k}: {(err / tol).max():.2f}x"

    def step(self, ins):
        for st, (kv, qn, qp), (w_uk, w_uv) in zip(self.layers, ins, self.w):
            st.run(kv, qn, qp, w_uk, w_uv)


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _tree_inputs(g, counts):
    parents, seen = [], []
    for n in counts:
        p = random_parents(g, n)
        parents += p
        seen.append(ancestors(p))
    return parents + [0] * (ROWS - len(parents)), seen


def _accept(g, counts, seen):
    """A random root-to-node path of each tree: counts and flat node lists."""
    start = np.concatenate([[0], np.cumsum(counts)])
    nodes, kept = np.zeros(ROWS, np.int32), []
    for b, n in enumerate(counts):
        path = np.flatnonzero(seen[b][int(g.integers(0, n))]) if n else []
        kept.append(len(path))
        nodes[start[b]:start[b] + len(path)] = path
    return kept, nodes


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
def test_serving_loop(cache):
    m = Model(cache, seed=3)
    # prompts, one sequence staying empty
    counts = [30, 70, 0, 1, 59]
    ins = m.inputs()
    m.plan.plan(_i32(counts))
    m.step(ins)
    torch.cuda.synchronize()
    m.check_out(ins, counts, [np.tril(np.ones((n, n), bool)) for n in counts])
    start = np.concatenate([[0], np.cumsum(counts)])
    for b, n in enumerate(counts):
        m.tokens[b] += [tuple(ins[k][0][start[b] + i] for k in range(2)) for i in range(n)]
    m.plan.keep_all()
    m.check_rows()
    for it in range(4):
        if it == 2:        # sequence 1 finishes, its pages return; sequence 2 gets a prompt beside others' trees
            m.plan.seq_lens[1] = 0
            m.tokens[1] = []
        counts = [int(m.g.integers(1, NODES + 1)) for _ in range(B)]
        counts[2] = 0 if it < 2 else 11
        counts[1] = 0 if it == 2 else counts[1]
        parents, seen = _tree_inputs(m.g, counts)
        ins = m.inputs()
        m.plan.plan(_i32(counts), _i32(parents))
        m.step(ins)
        torch.cuda.synchronize()
        m.check_out(ins, counts, seen)
        kept, nodes = _accept(m.g, counts, seen)
        m.plan.commit(m.layers, _i32(kept), _i32(nodes))
        start = np.concatenate([[0], np.cumsum(counts)])
        for b in range(B):
            path = nodes[start[b]:start[b] + kept[b]]
            m.tokens[b] += [tuple(ins[k][0][start[b] + int(i)] for k in range(2)) for i in path]
        m.check_rows()
        m.plan.check()
    # all finish: every page is free again
    m.plan.seq_lens.zero_()
    m.plan.plan(_i32([0] * B))
    m.plan.check()
    assert int(m.plan.free_count.item()) == m.plan.num_pages
    assert sorted(m.plan.free_pages.tolist()) == list(range(m.plan.num_pages))
    assert bool((m.plan.block_table == -1).all())


def test_one_graph_serves_every_step():
    """The whole step, plan to commit, recorded once and replayed; the same bits as eager calls."""
    eager, graph = Model("bf16", seed=4), Model("bf16", seed=4)
    counts0 = [64, 10, 128 - 74, 5, 1]
    for m in (eager, graph):
        m.ins = m.inputs()
        m.counts, m.parents, m.kept, m.nodes = _i32(counts0), _i32([0] * ROWS), _i32([0] * B), _i32([0] * ROWS)
        m.plan.plan(m.counts)
        m.step(m.ins)
        m.plan.keep_all()

    def body(m):
        m.plan.plan(m.counts, m.parents)
        m.step(m.ins)
        m.plan.commit(m.layers, m.kept, m.nodes)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    rec = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(rec, stream=side):
        body(graph)
    g = np.random.default_rng(9)
    for it in range(5):
        counts = [int(g.integers(0, NODES + 1)) for _ in range(B)]
        parents, seen = _tree_inputs(g, counts)
        kept, nodes = _accept(g, counts, seen)
        for m in (eager, graph):
            m.counts.copy_(_i32(counts))
            m.parents.copy_(_i32(parents))
            m.kept.copy_(_i32(kept))
            m.nodes.copy_(_i32(nodes))
            for dst, src in zip(m.ins, m.inputs()):
                for x, y in zip(dst, src):
                    x.copy_(y)
        body(eager)
        torch.cuda.synchronize()
        rec.replay()
        torch.cuda.synchronize()
        n = sum(counts)
        for a, b in zip(eager.layers, graph.layers):
            assert torch.equal(a.out[:n], b.out[:n]) and torch.equal(a.cache, b.cache)
        assert torch.equal(eager.plan.seq_lens, graph.plan.seq_lens)
        assert torch.equal(eager.plan.block_table, graph.plan.block_table)
    eager.plan.check()
    graph.plan.check()


def test_plan_that_does_not_fit_is_reported_and_harmless():
    m = Model("bf16", seed=5)
    m.plan.plan(_i32([60, 60, 0, 0, 0]))
    m.step(m.inputs())
    m.plan.keep_all()
    m.plan.check()
    before = m.layers[0].cache.clone()
    m.plan.plan(_i32([100, 100, 0, 0, 0]))            # more rows than max_rows
    m.step(m.inputs())
    m.plan.keep_all()
    with pytest.raises(RuntimeError, match="did not fit"):
        m.plan.check()
    assert torch.equal(before, m.layers[0].cache)
    assert m.plan.seq_lens.tolist() == [60, 60, 0, 0, 0]
    m.plan.check()                                    # cleared


def test_bounded_wait_leaves_the_next_call_sound():
    """A wait that runs out (the test hook withholds a query load) is flagged, and the next call is right."""
    m = Model("bf16", seed=6)
    m.plan.plan(_i32([40, 3, 0, 0, 7]))
    ins = m.inputs()
    m.step(ins)
    torch.cuda.synchronize()
    good = m.layers[0].out.clone()
    try:
        mla.mla_test_set_decode_wait(2_000_000, True)
        m.layers[0].attend()
        torch.cuda.synchronize()
    finally:
        mla.mla_test_set_decode_wait()
    assert int(m.plan.err.item()) & mla.MLA_DEVERR_TIMEOUT
    m.plan.err.zero_()
    m.layers[0].attend()
    m.layers[0].project_out(m.w[0][1])
    torch.cuda.synchronize()
    assert torch.equal(good[:50], m.layers[0].out[:50])
    m.plan.check()
