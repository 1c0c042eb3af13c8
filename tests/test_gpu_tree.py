"""The drafted-step operators on the GPU against plain 64-bit references:
mla_decode_tree, mla_step_plan, mla_cache_append_slots, mla_cache_commit."""
import math

import numpy as np
import pytest

import latent_attention_decode_absorbed_b200 as mla
from tree_ref import SCALE, Plan, ancestors, attend, commit_rows, pack_mask, page_table, random_parents

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
CODE = {"f32": mla.MLA_F32, "bf16": mla.MLA_BF16, "e4m3": mla.MLA_E4M3}


def _dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def make_pool(gen, num_pages, cache, rows_std=1.0):
    """Pool, row scales and the rows' values in float64 [num_pages*64, 576]."""
    x = torch.randn((num_pages * 64, 576), generator=gen, device="cuda") * rows_std
    if cache == "e4m3":
        x *= torch.rand((num_pages * 64, 1), generator=gen, device="cuda") * 1.5 + 0.5    # unequal row scales
        amax = x.abs().amax(1)
        codes = (x * (448.0 / amax)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        scale = (amax / 448.0).contiguous()
        vals = codes.double() * scale.double()[:, None]
        return mla.pack_cache_rows(codes.view(torch.uint8)), scale.view(num_pages, 64), vals
    x = x if cache == "f32" else x.to(torch.bfloat16)
    return mla.pack_cache_rows(x), None, x.double()


class Problem:
    """Inputs of one mla_decode_tree call.  mask: 'tree', 'chain' (no mask
    given), 'chain_mask' (a chain as masks) or 'random' (any bits)."""

    def __init__(self, cache, H, counts, prefix, mask="tree", seed=0, q_std=0.6, pad=3, words=None, o_dtype=None,
                 bad_pages=()):
        g = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.cache, self.H, self.counts = cache, H, list(counts)
        self.B, self.N = len(counts), int(sum(counts))
        self.rows = self.N + pad
        self.lens = [p + n for p, n in zip(prefix, counts)]
        self.bt, self.num_pages = page_table(self.lens, 2, g, max(1, max(-(-x // 64) for x in self.lens)) + 1)
        self.pool, self.scale, self.vals = make_pool(gen, self.num_pages, cache)
        self.start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.words = words or max(1, -(-max(counts) // 64))
        self.seen, packed = [], np.zeros((self.rows, self.words), np.int64)
        for b, n in enumerate(counts):
            if mask in ("chain", "chain_mask"):
                s = np.tril(np.ones((n, n), bool))
            elif mask == "random":
                s = g.random((n, n)) < 0.3
            else:
                s = ancestors(random_parents(g, n, roots=int(g.integers(1, 3))))
            self.seen.append(s)
            full = np.ones((n, 64 * self.words), bool)      # bits past the last drafted row are set and ignored
            full[:, :min(n, 64 * self.words)] = s[:, :64 * self.words]
            packed[self.start[b]:self.start[b] + n] = pack_mask(full, self.words)
        self.mask = None if mask == "chain" else _dev(packed)
        for b, k in bad_pages:
            self.bt[b, k] = [-1, self.num_pages][k % 2]
        self.bad = set(bad_pages)
        qdt = torch.float32 if cache == "f32" else torch.bfloat16
        self.q = (torch.randn((self.rows, H, 576), generator=gen, device="cuda") * q_std).to(qdt)
        self.o_dtype = o_dtype or ("f32" if cache == "f32" else "bf16")
        odt = torch.float32 if self.o_dtype == "f32" else torch.bfloat16
        self.o = torch.full((self.rows, H, 512), 7.0, device="cuda", dtype=odt)
        self.lse = torch.full((self.rows, H), 7.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(max(16, mla.mla_decode_tree_workspace_bytes(CODE[cache], self.rows, H)),
                              dtype=torch.uint8, device="cuda")
        self.ws.fill_(0xFF)                                 # NaN patterns: nothing may depend on old contents
        self.table, self.kv_lens, self.row_start = _dev(self.bt), _dev(np.array(self.lens, np.int32)), _dev(self.start)

    def run(self, stream=None, **over):
        a = dict(q_abs=self.q, q_dtype=mla.MLA_F32 if self.cache == "f32" else mla.MLA_BF16, cache=self.pool,
                 cache_scale=self.scale, cache_dtype=CODE[self.cache], num_pages=self.num_pages,
                 block_table=self.table, max_pages_per_seq=self.bt.shape[1], page_size=64, kv_lens=self.kv_lens,
                 row_start=self.row_start, batch=self.B, max_rows=self.rows, n_heads=self.H, tree_mask=self.mask,
                 mask_words=self.words, softmax_scale=SCALE, workspace=self.ws, o_lat=self.o,
                 o_dtype=CODE[self.o_dtype], lse_out=self.lse, err_word=self.err, stream=stream)
        a.update(over)
        mla.mla_decode_tree(**a)

    def check(self):
        torch.cuda.synchronize()
        o, lse = self.o.double(), self.lse.double()
        pad = self.N
        assert bool((o[pad:] == 7.0).all()) and bool((lse[pad:] == 7.0).all()), "rows behind the last sequence changed"
        for b in range(self.B):
            n, L = self.counts[b], self.lens[b]
            if n == 0:
                continue
            slots = np.concatenate([np.arange(64) + 64 * max(0, min(int(x), self.num_pages - 1))
                                    for x in self.bt[b, :-(-L // 64)]])[:L]
            rows = self.vals[_dev(slots)]
            visible = np.ones(L, bool)
            for bb, k in self.bad:
                if bb == b:
                    visible[64 * k:64 * k + 64] = False
            for i in range(n):
                seen = visible.copy()
                s = self.seen[b][i].copy()
                s[64 * self.words:] = False
                if self.mask is None:
                    s = self.seen[b][i]
                seen[L - n:] &= s
                r = int(self.start[b]) + i
                ref, rl, a, l = attend(self.q[r].double(), rows, _dev(seen))
                self._close(r, o[r], lse[r], ref, rl, a, l, rows, _dev(seen))

    def _close(self, r, o, lse, ref, rl, a, l, rows, seen):
        empty = torch.isinf(rl)
        assert bool((lse[empty] == -math.inf).all()) and bool((o[empty] == 0).all()), f"row {r}: an empty row"
        if bool(empty.all()):
            return
        q, x = self.q[r].double(), rows[seen]
        # scores: 576 products summed in fp32 (each addition at most a full step 2^-23 of the running sum of
        # magnitudes off, tensor cores truncate), the scales three more roundings
        mag = SCALE * (q.abs() @ x.abs().T).amax(1)
        e_s = 580 * 2.0 ** -23 * mag
        if self.cache == "e4m3":     # query components under 2^-9 of the largest: 2^-17 of the largest off
            e_s = e_s + SCALE * 2.0 ** -17 * q.abs().amax(1) * x.abs().sum(1).amax()
        # statistics: ex2 / exp 2^-21 per weight, fp32 sums of up to len(x) terms in runs of 64
        e_l = e_s + 2.0 ** -20 * (1 + rl.abs())
        assert bool(((lse - rl).abs() <= e_l).all()), \
            f"row {r}: lse off by {(lse - rl).abs().max():.3e}, allowed {e_l.min():.3e}"
        w = {"f32": 2.0 ** -20, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -8}[self.cache]     # rounding of a weight
        tol = (w + 2 * e_s[:, None] + 2.0 ** -18) * a
        if self.cache == "e4m3":
            # weights are carried as p * 16 * scale / reference; what lies below e4m3's last step (2^-9) is lost:
            # at most 2^-10 / 16 of the reference scale per row, and the reference is at most the largest scale
            scale = (x.abs().amax(1) / 448.0).amax()
            codes = (x[:, :512].abs() / (x.abs().amax(1, keepdim=True) / 448.0)).sum(0)
            tol = tol + 2.0 ** -14 * scale * codes[None] / l[:, None]
        tol = tol + (2.0 ** -8 if self.o_dtype == "bf16" else 2.0 ** -22) * ref.abs() + 1e-30
        bad = (o - ref).abs() > tol
        assert not bool(bad.any()), f"row {r}: {int(bad.sum())} outputs off, worst {((o - ref).abs() / tol).max():.2f}x"


CASES = [
    # (id, cache, heads, counts, prefix, mask)
    ("one_row", "bf16", 128, [1], [0], "tree"),
    ("one_token", "bf16", 128, [1], [300], "chain"),
    ("long_one", "bf16", 128, [1], [5000], "tree"),
    ("ragged", "bf16", 128, [5, 0, 9, 1, 16], [70, 40, 0, 511, 255], "tree"),
    ("ends_in_page", "bf16", 128, [3, 64, 7], [61, 64, 57], "random"),
    ("empty_rows", "bf16", 96, [6, 4], [0, 0], "random"),
    ("heads16", "bf16", 16, [8, 9, 7, 30], [1000, 63, 128, 2000], "tree"),
    ("heads1", "bf16", 1, [200, 3], [700, 1], "random"),
    ("heads3_chain", "bf16", 3, [50, 11], [77, 900], "chain"),
    ("heads65", "bf16", 65, [2, 3, 4], [190, 191, 192], "chain_mask"),
    ("wide_tree", "bf16", 32, [130, 65], [33, 400], "random"),
    ("many_seqs", "bf16", 24, [1 + (7 * i) % 5 for i in range(400)], [(37 * i) % 300 for i in range(400)], "tree"),
    ("dealt_out", "bf16", 128, [1 + (5 * i) % 9 for i in range(30)], [(211 * i) % 1500 for i in range(30)], "tree"),
    ("whole_columns", "bf16", 128, [1 + i % 2 for i in range(90)], [300 + (53 * i) % 200 for i in range(90)], "tree"),
    ("whole_columns_fewer_rows", "e4m3", 128, [1 + i % 2 for i in range(40)], [300 + (53 * i) % 200 for i in range(40)],
     "tree"),
    ("more_seqs_than_dealt", "bf16", 40, [1 + i % 2 for i in range(1100)], [(37 * i) % 300 for i in range(1100)],
     "chain"),
    ("split_tiles", "bf16", 128, [20, 20], [3000, 9000], "tree"),
    ("e4m3_one", "e4m3", 128, [1], [0], "tree"),
    ("e4m3_ragged", "e4m3", 128, [5, 0, 9, 1], [70, 40, 0, 2500], "tree"),
    ("e4m3_heads16", "e4m3", 16, [8, 33], [1000, 63], "random"),
    ("e4m3_split", "e4m3", 128, [12, 3], [6000, 700], "random"),
    ("e4m3_wide", "e4m3", 7, [130], [129], "tree"),
    ("f32_one", "f32", 16, [1], [0], "tree"),
    ("f32_ragged", "f32", 16, [5, 0, 9, 1], [70, 40, 0, 700], "tree"),
    ("f32_random", "f32", 33, [4, 70], [0, 31], "random"),
    ("f32_chain", "f32", 5, [3], [2000], "chain"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: c[0])
def test_tree_attention(case):
    name, cache, H, counts, prefix, mask = case
    p = Problem(cache, H, counts, prefix, mask, seed=sum(map(ord, name)))
    p.run()
    p.check()
    assert int(p.err.item()) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
def test_sharp_scores_and_fp32_output(cache):
    """Scores of standard deviation 10 (the running maximum moves many times), o_lat in fp32."""
    p = Problem(cache, 48, [7, 3], [1500, 200], "tree", seed=5, q_std=6.0, o_dtype="f32")
    p.run()
    p.check()


def test_mask_words_short_of_the_tree():
    """Drafted rows past the mask's words are not seen."""
    p = Problem("bf16", 16, [100, 70], [40, 10], "random", seed=6, words=1)
    p.run()
    p.check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "f32"])
def test_pages_outside_the_pool_are_not_seen(cache):
    p = Problem(cache, 16, [4, 5], [500, 130], "tree", seed=7, bad_pages=[(0, 2), (0, 3), (1, 1)])
    p.run()
    p.check()
    assert int(p.err.item()) == mla.MLA_DEVERR_PAGE


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_rows_behind_the_end_do_not_count(cache):
    """Large finite rows behind the end of a sequence and behind a mask change no bit."""
    a = Problem(cache, 64, [6, 3], [100, 30], "tree", seed=8)
    a.run()
    torch.cuda.synchronize()
    first = a.o.clone()
    rows = mla.unpack_cache_rows(a.pool).clone()
    for b in range(2):
        L = a.lens[b]
        last = int(a.bt[b, (L - 1) // 64])
        stale = slice(last * 64 + (L - 1) % 64 + 1, last * 64 + 64)
        rows[stale] = 0x7E if cache == "e4m3" else 3e4     # e4m3: 448
        if cache == "e4m3":
            a.scale.view(-1)[stale] = 1e3
    a.pool.copy_(mla.pack_cache_rows(rows))
    a.run()
    torch.cuda.synchronize()
    assert torch.equal(first, a.o)


def test_f32_hidden_rows_may_hold_anything():
    """NaN and infinities in rows that no node sees change no bit over an fp32 cache."""
    p = Problem("f32", 20, [6, 3], [100, 30], "tree", seed=17)
    for b in range(2):                                 # the last drafted row is seen by nobody
        n, s = p.counts[b], p.seen[b]
        s[:, n - 1] = False
        p.mask[int(p.start[b]):int(p.start[b]) + n, 0] = _dev(pack_mask(s, 1))[:, 0]
    p.run()
    torch.cuda.synchronize()
    first, lse = p.o.clone(), p.lse.clone()
    rows = mla.unpack_cache_rows(p.pool).clone()
    for b in range(2):
        L = p.lens[b]
        last = int(p.bt[b, (L - 1) // 64]) * 64
        rows[last + (L - 1) % 64] = float("nan")
        rows[last + (L - 1) % 64 + 1:last + 64] = float("inf")
    p.pool.copy_(mla.pack_cache_rows(rows))
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(first, p.o) and torch.equal(lse, p.lse)
    assert not bool(torch.isnan(p.o).any())


def test_same_bits_again_and_on_another_stream():
    p = Problem("bf16", 128, [20, 7, 33], [3000, 500, 900], "tree", seed=9)
    p.run()
    torch.cuda.synchronize()
    o, lse = p.o.clone(), p.lse.clone()
    side = torch.cuda.Stream()
    for k in range(3):
        p.o.fill_(7.0)
        p.ws.fill_(0x5A + k)
        torch.cuda.synchronize()
        p.run(stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o, p.o) and torch.equal(lse, p.lse)


def test_impossible_sequences_are_skipped():
    p = Problem("bf16", 16, [4, 4, 4], [100, 100, 100], "tree", seed=10)
    p.run()
    torch.cuda.synchronize()
    good = p.o.clone()
    p.o.fill_(7.0)
    p.kv_lens[1] = 3                                   # fewer cached rows than drafted ones
    p.run()
    torch.cuda.synchronize()
    assert int(p.err.item()) == mla.MLA_DEVERR_POSITION
    assert torch.equal(p.o[:4], good[:4]) and torch.equal(p.o[8:12], good[8:12])
    assert bool((p.o[4:8] == 7.0).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("start", [[0, 8, 4, 12], [0, 4, 8, 99], [-1, 4, 8, 12], [0, 12, 0, 12]])
def test_row_offsets_out_of_order_compute_nothing(start, cache):
    p = Problem(cache, 16, [4, 4, 4], [100, 100, 100], "tree", seed=13)
    p.row_start.copy_(_dev(np.array(start, np.int32)))
    p.run()
    torch.cuda.synchronize()
    assert int(p.err.item()) & mla.MLA_DEVERR_POSITION
    assert bool((p.o == 7.0).all()) and bool((p.lse == 7.0).all())


def test_captured_call_follows_device_lengths():
    """One captured graph serves other lengths, row counts, masks and tables."""
    a = Problem("bf16", 128, [8, 8], [2000, 110], "tree", seed=11)
    b = Problem("bf16", 128, [3, 13], [50, 1990], "tree", seed=12)
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = b.o.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        a.run()
    # b's problem in a's buffers
    assert b.num_pages <= a.num_pages and b.bt.shape == a.bt.shape
    a.pool[:b.num_pages].copy_(b.pool)
    for x, y in ((a.q, b.q), (a.mask, b.mask), (a.table, b.table), (a.kv_lens, b.kv_lens),
                 (a.row_start, b.row_start)):
        x.copy_(y)
    a.o.fill_(7.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.o, want)


# ------------------------------------------------------------------ step plan
def _plan_case(seed, B, lens, counts, held_extra=None, tree=True, words=1, spare=5, pad=4, width_extra=1):
    g = np.random.default_rng(seed)
    need = [-(-(l + n) // 64) for l, n in zip(lens, counts)]
    held = [-(-l // 64) for l in lens]
    if held_extra:
        held = [h + e for h, e in zip(held, held_extra)]
    width = max(1, max(need + held)) + width_extra
    take = sum(max(0, n - h) for n, h in zip(need, held))
    num_pages = sum(held) + take + spare
    ids = g.permutation(num_pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = np.full(num_pages, -1, np.int32)
    free[:num_pages - at] = ids[at:]
    parents = None
    if tree:
        parents = np.array([p for n in counts for p in random_parents(g, n, roots=int(g.integers(1, 3)))] + [0] * pad,
                           np.int32)
    return dict(lens=lens, counts=counts, held=held, table=table, free=free, free_count=num_pages - at,
                num_pages=num_pages, parents=parents, words=words, max_rows=sum(counts) + pad)


def _run_plan(c, in_place=True, mask=True, max_rows=None, parents=True):
    B = len(c["lens"])
    R = c["max_rows"] if max_rows is None else max_rows
    i32 = lambda *s: torch.full(s, -77, dtype=torch.int32, device="cuda")  # noqa: E731
    d = dict(lens=_dev(np.array(c["lens"], np.int32)), counts=_dev(np.array(c["counts"], np.int32)),
             held=_dev(np.array(c["held"], np.int32)), table=_dev(c["table"]), free=_dev(c["free"]),
             free_count=_dev(np.array([c["free_count"]], np.int32)), row_start=i32(B + 1), kv_lens=i32(B),
             seq_ids=i32(R), positions=i32(R), slots=i32(R), err=torch.zeros(1, dtype=torch.int32, device="cuda"),
             mask=torch.full((R, c["words"]), -77, dtype=torch.int64, device="cuda") if mask else None)
    d["held_out"] = d["held"] if in_place else i32(B)
    d["free_count_out"] = d["free_count"] if in_place else i32(1)
    par = _dev(c["parents"]) if parents and c["parents"] is not None else None
    mla.mla_step_plan(d["lens"], d["counts"], par, B, R, c["words"], d["held"], d["held_out"], d["free"],
                      d["free_count"], d["free_count_out"], d["table"], c["table"].shape[1], 64, c["num_pages"],
                      d["row_start"], d["kv_lens"], d["seq_ids"], d["positions"], d["slots"], d["mask"], d["err"])
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() if v is not None else None for k, v in d.items()}


def _same_plan(got, c, ref, mask=True):
    np.testing.assert_array_equal(got["table"], ref.table)
    np.testing.assert_array_equal(got["free"], ref.free)
    np.testing.assert_array_equal(got["held_out"], ref.held)
    assert int(got["free_count_out"][0]) == ref.free_count
    np.testing.assert_array_equal(got["row_start"], ref.row_start)
    np.testing.assert_array_equal(got["kv_lens"], ref.kv_lens)
    np.testing.assert_array_equal(got["seq_ids"], ref.seq_ids)
    np.testing.assert_array_equal(got["slots"], ref.slots)
    np.testing.assert_array_equal(got["positions"], ref.positions)
    if mask:
        np.testing.assert_array_equal(got["mask"], ref.mask)
    assert int(got["err"][0]) == 0


PLANS = [
    ("one", 1, [0], [1], None, True, 1),
    ("nothing_new", 3, [64, 0, 5], [0, 0, 0], None, True, 1),
    ("small", 4, [63, 64, 65, 0], [1, 1, 1, 130], None, True, 3),
    ("releases", 6, [0, 200, 64, 10, 0, 500], [0, 3, 64, 2, 7, 20], [4, 0, 2, 3, 0, 0], True, 1),
    ("prompts", 5, [0] * 5, [1000, 1, 64, 2500, 777], None, False, 0),
    ("mixed", 3, [100, 0, 4000], [1, 900, 1], None, False, 0),
    ("chain_masks", 3, [5, 60, 0], [70, 3, 1], None, False, 2),
    ("many", 2500, [(37 * i) % 200 for i in range(2500)], [(5 * i) % 9 for i in range(2500)],
     [(3 * i) % 4 for i in range(2500)], True, 1),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("case", PLANS, ids=lambda c: c[0])
def test_step_plan(case, in_place):
    name, B, lens, counts, extra, tree, words = case
    c = _plan_case(len(name), B, lens, counts, extra, tree, words)
    ref = Plan(lens, counts, c["held"], c["table"], c["free"], c["free_count"], c["num_pages"], c["parents"], words,
               c["max_rows"])
    _same_plan(_run_plan(c, in_place, mask=words > 0), c, ref, mask=words > 0)


@pytest.mark.parametrize("what", ["pages", "rows", "table", "mask", "length", "count", "held", "free_count"])
def test_step_plan_that_does_not_fit_changes_nothing(what):
    c = _plan_case(3, 4, [100, 5, 640, 0], [20, 60, 3, 30], None, True, 1)
    rows, flag = None, mla.MLA_DEVERR_CAPACITY
    if what == "pages":
        c["free_count"] = 1
    elif what == "rows":
        rows = 112
    elif what == "table":
        c["lens"] = [100, 5, 64 * c["table"].shape[1] - 1, 0]
    elif what == "mask":
        c["counts"] = [20, 65, 3, 20]
    else:
        flag = mla.MLA_DEVERR_POSITION
        if what == "length":
            c["lens"] = [100, -1, 640, 0]
        elif what == "count":
            c["counts"] = [20, 60, -3, 30]
        elif what == "held":
            c["held"] = [c["held"][0], c["table"].shape[1] + 1, c["held"][2], 0]
        else:
            c["free_count"] = c["num_pages"] + 1
    got = _run_plan(c, max_rows=rows)
    assert int(got["err"][0]) & flag
    np.testing.assert_array_equal(got["table"], c["table"])
    np.testing.assert_array_equal(got["free"], c["free"])
    np.testing.assert_array_equal(got["held_out"], c["held"])
    assert int(got["free_count_out"][0]) == c["free_count"]
    assert not got["row_start"].any()
    np.testing.assert_array_equal(got["kv_lens"], c["lens"])
    assert (got["slots"] == -1).all() and (got["seq_ids"] == -1).all()


def test_step_plan_flags_a_parent_that_follows_its_child():
    c = _plan_case(4, 1, [10], [4], None, True, 1, pad=0)
    c["parents"] = np.array([-1, 0, 3, 1], np.int32)
    got = _run_plan(c)
    assert int(got["err"][0]) == mla.MLA_DEVERR_POSITION
    np.testing.assert_array_equal(got["mask"][:, 0], [1, 3, 4, 11])
    np.testing.assert_array_equal(got["positions"], [10, 11, 10, 12])


# ------------------------------------------------------------------ append by slot
@pytest.mark.parametrize("cache", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("kv", ["f32", "bf16"])
def test_append_slots_writes_the_append_s_bits(cache, kv):
    """At the slots a block table gives, the same bits as mla_cache_append; padding and bad rows skipped."""
    g = np.random.default_rng(1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    n, num_pages, max_pos = 300, 9, 500
    bt = g.permutation(num_pages)[:6].astype(np.int32).reshape(1, 6)
    pos = g.permutation(6 * 64)[:n].astype(np.int32)
    x = torch.randn((n, 576), generator=gen, device="cuda").to(torch.float32 if kv == "f32" else torch.bfloat16)
    gain = 1 + 0.1 * torch.randn(512, generator=gen, device="cuda")
    cos = np.empty((max_pos, 32), np.float32)
    sin = np.empty_like(cos)
    mla.mla_rope_table(10000.0, max_pos, cos, sin)
    cos, sin = _dev(cos), _dev(sin)
    tdt = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}[cache]
    new = lambda: (torch.zeros((num_pages, 9, 64, 64), dtype=tdt, device="cuda"),  # noqa: E731
                   torch.zeros((num_pages, 64), device="cuda") if cache == "e4m3" else None)
    (a, sa), (b, sb) = new(), new()
    mla.mla_cache_append(x, CODE[kv], n, torch.zeros(n, dtype=torch.int32, device="cuda"), _dev(pos), _dev(bt), 1, 6,
                         64, gain, 1e-6, cos, sin, max_pos, a, sa, CODE[cache], num_pages)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = (bt[0, pos // 64] * 64 + pos % 64).astype(np.int32)
    more = np.array([-1, -1, -2, num_pages * 64, 3, 3], np.int32)       # padding twice, outside twice, bad positions
    xp = torch.cat([x, x[:6]])
    mla.mla_cache_append_slots(xp, CODE[kv], n + 4, _dev(np.concatenate([slots, more])),
                               _dev(np.concatenate([pos, np.zeros(4, np.int32), np.array([-1, max_pos], np.int32)])),
                               gain, 1e-6, cos, sin, max_pos, b, sb, CODE[cache], num_pages, err)
    torch.cuda.synchronize()
    assert int(err.item()) == mla.MLA_DEVERR_PAGE
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert sa is None or torch.equal(sa, sb)
    err.zero_()
    mla.mla_cache_append_slots(x, CODE[kv], 2, _dev(np.array([0, 1], np.int32)),
                               _dev(np.array([-1, max_pos], np.int32)), gain, 1e-6, cos, sin, max_pos, b, sb,
                               CODE[cache], num_pages, err)
    torch.cuda.synchronize()
    assert int(err.item()) == mla.MLA_DEVERR_POSITION
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("cache", ["f32", "bf16", "e4m3"])
def test_commit(cache):
    """Paths that overlap their targets, none, all, long ones; every other row keeps its bits."""
    g = np.random.default_rng(2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    n = [1, 8, 0, 16, 200, 200, 64, 5]
    prefix = [0, 60, 10, 127, 300, 0, 64, 1000]
    counts = [1, 4, 0, 0, 150, 200, 1, 3]
    B = len(n)
    lens = [p + k for p, k in zip(prefix, n)]
    bt, num_pages = page_table(lens, 2, g)
    pool, scale, _ = make_pool(gen, num_pages, cache)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    nodes = np.full(start[-1], -5, np.int32)
    for b in range(B):
        nodes[start[b]:start[b] + counts[b]] = np.sort(g.permutation(n[b])[:counts[b]])
    before = mla.unpack_cache_rows(pool).contiguous().view(torch.uint8).cpu().numpy().reshape(num_pages * 64, -1)
    sc = None if scale is None else scale.view(-1).cpu().numpy().copy()
    want, want_lens = commit_rows(before, bt, lens, start, counts, nodes)
    out = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (_dev(np.array(lens, np.int32)), _dev(start), B, int(start[-1]), _dev(np.array(counts, np.int32)),
            _dev(nodes), _dev(bt), bt.shape[1], 64, pool, scale, CODE[cache], num_pages, out, err)
    mla.mla_cache_commit(*args)
    torch.cuda.synchronize()
    got = mla.unpack_cache_rows(pool).contiguous().view(torch.uint8).cpu().numpy().reshape(num_pages * 64, -1)
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(out.cpu().numpy(), want_lens)
    if sc is not None:
        np.testing.assert_array_equal(scale.view(-1).cpu().numpy(), commit_rows(sc, bt, lens, start, counts, nodes)[0])
    assert int(err.item()) == 0


@pytest.mark.parametrize("path", [[3, 2], [0, 0], [-1, 2], [0, 8], None])
def test_commit_refuses_a_path_that_is_none(path):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    pool, _, _ = make_pool(gen, 4, "bf16")
    before = pool.clone()
    nodes = np.zeros(8, np.int32)
    count = 9 if path is None else len(path)
    if path:
        nodes[:len(path)] = path
    out = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_commit(_dev(np.array([108], np.int32)), _dev(np.array([0, 8], np.int32)), 1, 8,
                         _dev(np.array([count], np.int32)), _dev(nodes), _dev(np.array([[2, 0]], np.int32)), 2, 64,
                         pool, None, mla.MLA_BF16, 4, out, err)
    torch.cuda.synchronize()
    assert int(err.item()) == mla.MLA_DEVERR_POSITION
    assert int(out.item()) == 100 and torch.equal(pool, before)


def test_commit_skips_rows_outside_the_pool():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    pool, _, _ = make_pool(gen, 4, "bf16")
    before = pool.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.mla_cache_commit(_dev(np.array([68], np.int32)), _dev(np.array([0, 8], np.int32)), 1, 8,
                         _dev(np.array([2], np.int32)), _dev(np.array([1, 7] + [0] * 6, np.int32)),
                         _dev(np.array([[2, 4]], np.int32)), 2, 64, pool, None, mla.MLA_BF16, 4, None, err)
    torch.cuda.synchronize()
    assert int(err.item()) == mla.MLA_DEVERR_PAGE
    rows, old = mla.unpack_cache_rows(pool), mla.unpack_cache_rows(before)
    assert torch.equal(rows[2 * 64 + 60], old[2 * 64 + 61])
    rows[2 * 64 + 60] = old[2 * 64 + 60]
    assert torch.equal(rows, old)


# ------------------------------------------------------------------ far pages, two calls at once
def test_pages_past_32_bit_offsets():
    """A pool of more than 2^32 bytes and 2^31 numbers: attention, append and commit at its far end."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(14)
    num_pages, far = 60000, 59000
    pool = torch.empty((num_pages, 9, 64, 64), dtype=torch.bfloat16, device="cuda")
    pool[0].zero_()
    p = Problem("bf16", 16, [5, 3], [200, 70], "tree", seed=14)
    pool[far:far + p.num_pages].copy_(p.pool)
    table = torch.where(p.table >= 0, p.table + far, p.table)
    p.run(cache=pool, num_pages=num_pages, block_table=table)
    p.check()
    assert int(p.err.item()) == 0
    # append by slot: the same bits as near the pool's start
    n, max_pos = 100, 256
    x = torch.randn((n, 576), generator=gen, device="cuda").to(torch.bfloat16)
    cos = np.empty((max_pos, 32), np.float32)
    sin = np.empty_like(cos)
    mla.mla_rope_table(10000.0, max_pos, cos, sin)
    cos, sin = _dev(cos), _dev(sin)
    slots = torch.randperm(128, generator=gen, device="cuda")[:n].int()
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    near = torch.zeros((2, 9, 64, 64), dtype=torch.bfloat16, device="cuda")
    pool[far:far + 2].zero_()
    for dst, off in ((near, 0), (pool, far * 64)):
        mla.mla_cache_append_slots(x, mla.MLA_BF16, n, slots + off, pos, None, 1e-6, cos, sin, max_pos, dst, None,
                                   mla.MLA_BF16, dst.shape[0])
    assert torch.equal(pool[far:far + 2], near)
    # commit: the same rows
    lens, start = _dev(np.array([110], np.int32)), _dev(np.array([0, 20], np.int32))
    counts, nodes = _dev(np.array([3], np.int32)), _dev(np.array([1, 7, 19] + [0] * 17, np.int32))
    for dst, t in ((near, [[1, 0]]), (pool, [[far + 1, far]])):
        mla.mla_cache_commit(lens, start, 1, 20, counts, nodes, _dev(np.array(t, np.int32)), 2, 64, dst, None,
                             mla.MLA_BF16, dst.shape[0])
    torch.cuda.synchronize()
    assert torch.equal(pool[far:far + 2], near)


def test_two_calls_at_once_on_two_streams():
    """Calls with workspaces of their own on two streams give each its own result."""
    a = Problem("bf16", 128, [9, 4], [1500, 900], "tree", seed=15)
    b = Problem("e4m3", 64, [12, 3, 8], [700, 64, 2000], "random", seed=16)
    want = []
    for p in (a, b):
        p.run()
        torch.cuda.synchronize()
        want.append((p.o.clone(), p.lse.clone()))
        p.o.fill_(7.0)
        p.lse.fill_(7.0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(stream=s1)
        b.run(stream=s2)
    torch.cuda.synchronize()
    for p, (o, lse) in zip((a, b), want):
        assert torch.equal(p.o, o) and torch.equal(p.lse, lse)
