"""Cases of a drafted (speculative) decode step over the paged latent cache.

Four operators make up such a step around the attention of one layer:

  plan     mla_step_plan           request lengths and drafted trees -> pages, block table, slot map,
                                   positions and ancestor masks
  append   mla_cache_append_slots  the drafted tokens' rows written at the planned slots
  tree     mla_decode_tree         attention of every drafted token over its sequence's cached rows and
                                   its own ancestors in the tree
  commit   mla_cache_commit        the rows of the accepted path moved to the front of the drafted rows

``run`` computes each in plain torch operations, or, with ``own`` true, with the library's calls.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D_C, D_R, D_ROW, PAGE = 512, 64, 576, 64
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
# the largest drawn attention: drafted tokens x heads x cached rows, and cached rows, padded to the longest sequence
MOST_SCORES, MOST_ROWS = 1 << 30, 1 << 20


def listed():
    return [
        # a sequence's next token with nothing drafted: the latency of one request
        dict(name="tree_one_token", op="tree", batch=1, heads=128, nodes_lo=1, nodes_hi=1, len_lo=4096, len_hi=4096,
             cache="bf16"),
        # a small fp32 model checking four drafted tokens
        dict(name="tree_f32_small", op="tree", batch=1, heads=16, nodes_lo=4, nodes_hi=4, len_lo=256, len_hi=256,
             cache="f32"),
        # one GPU's sixteen heads of a head-sharded model, trees of eight over a serving batch
        dict(name="tree_sharded_heads", op="tree", batch=64, heads=16, nodes_lo=8, nodes_hi=8, len_lo=1024,
             len_hi=8192, cache="bf16"),
        # a serving batch of ragged lengths with trees of 5 to 16 drafted tokens
        dict(name="tree_serving", op="tree", batch=64, heads=128, nodes_lo=5, nodes_hi=16, len_lo=1024, len_hi=8192,
             cache="bf16"),
        # two long documents with a tree of 32 each
        dict(name="tree_long", op="tree", batch=2, heads=128, nodes_lo=32, nodes_hi=32, len_lo=131072,
             len_hi=131072, cache="bf16"),
        # many sequences over an 8-bit cache, two to six drafted tokens each
        dict(name="tree_e4m3", op="tree", batch=128, heads=128, nodes_lo=2, nodes_hi=6, len_lo=2048, len_hi=4096,
             cache="e4m3"),
        # a decode step's bookkeeping: a tree of 16 for each of 64 sequences
        dict(name="plan_trees", op="plan", batch=64, nodes_lo=16, nodes_hi=16, len_lo=1024, len_hi=8192, tree=True),
        # whole prompts admitted at once: 256 requests of up to 8192 tokens
        dict(name="plan_prompts", op="plan", batch=256, nodes_lo=64, nodes_hi=8192, len_lo=0, len_hi=0, tree=False),
        # the drafted rows of a serving batch
        dict(name="append_trees", op="append", rows=1024, cache="bf16"),
        # the rows of admitted prompts into an 8-bit cache
        dict(name="append_prompts", op="append", rows=65536, cache="e4m3"),
        # the accepted paths of a serving batch
        dict(name="commit_serving", op="commit", batch=64, nodes=16, count_hi=5, length=4096, cache="bf16"),
        # a large batch over an 8-bit cache
        dict(name="commit_e4m3", op="commit", batch=512, nodes=32, count_hi=8, length=1024, cache="e4m3"),
    ]


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["tree", "tree", "tree", "plan", "append", "commit"])
    if op == "tree":
        cache = rng.choice(["bf16", "bf16", "e4m3", "f32"])
        if cache == "f32":      # the fp32 form serves small models
            nodes = _log_int(rng, 1, 16)
            length = _log_int(rng, 16, 2048)
            return dict(op=op, batch=_log_int(rng, 1, 8), heads=rng.randint(1, 32), nodes_lo=max(1, nodes // 2),
                        nodes_hi=nodes, len_lo=(length + 1) // 2, len_hi=length, cache=cache)
        batch, heads = _log_int(rng, 1, 128), rng.choice([8, 16, 32, 64, 128, rng.randint(1, 128)])
        nodes, length = _log_int(rng, 1, 64), _log_int(rng, 64, 131072)
        while (batch * heads * nodes * (length + 2 * PAGE + nodes) > MOST_SCORES or batch * length > MOST_ROWS):
            if batch > 1 and rng.random() < 0.5:
                batch = (batch + 1) // 2
            elif nodes > 1 and rng.random() < 0.5:
                nodes = (nodes + 1) // 2
            else:
                length = max(64, (length + 1) // 2)
        return dict(op=op, batch=batch, heads=heads, nodes_lo=max(1, nodes // 3), nodes_hi=nodes,
                    len_lo=max(1, length // rng.choice([1, 4, 8])), len_hi=length, cache=cache)
    if op == "plan":
        if rng.random() < 0.5:
            nodes = _log_int(rng, 1, 128)
            length = _log_int(rng, 64, 32768)
            return dict(op=op, batch=_log_int(rng, 1, 1024), nodes_lo=max(1, nodes // 2), nodes_hi=nodes,
                        len_lo=length // 8, len_hi=length, tree=True)
        return dict(op=op, batch=_log_int(rng, 1, 256), nodes_lo=_log_int(rng, 1, 64),
                    nodes_hi=_log_int(rng, 64, 8192), len_lo=0, len_hi=0, tree=False)
    if op == "append":
        return dict(op=op, rows=_log_int(rng, 1, 65536), cache=rng.choice(["bf16", "e4m3", "f32"]))
    return dict(op=op, batch=_log_int(rng, 1, 512), nodes=rng.randint(16, 40), count_hi=rng.randint(1, 8),
                length=_log_int(rng, 64, 4096), cache=rng.choice(["bf16", "e4m3", "f32"]))


# ------------------------------------------------------------------ inputs
def _spread(lo: int, hi: int, n: int):
    """n whole numbers spread evenly over [lo, hi]."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _shuffled(values, seed: int, tag: int):
    out = list(values)
    random.Random(seed * 16 + tag).shuffle(out)
    return out


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _tree(n: int, rng: random.Random):
    """Parents of a drafted tree of n nodes in breadth-first order, node 0 the root."""
    parents = [-1]
    for i in range(1, n):
        parents.append(rng.randint(max(0, (i - 1) // 3 - 1), max(0, (i - 1) // 2)))
    return parents


def _ancestor_words(parents, words: int):
    """Bit k of node i: k is i or an ancestor of i; as `words` signed 64-bit numbers per node."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | (1 << i))
    low = (1 << 64) - 1
    split = [[(b >> (64 * w)) & low for w in range(words)] for b in bits]
    return [[v - (1 << 64) if v >> 63 else v for v in row] for row in split]


def _pool_rows(num_pages: int, cache: str, gen):
    """A page-blocked pool [num_pages, 9, 64, 64] of rows as the append leaves them, and its row scales."""
    x = torch.randn((num_pages, 9, PAGE, 64), generator=gen, device="cuda", dtype=torch.float32)
    if cache == "f32":
        return x, None
    if cache == "bf16":
        return x.to(torch.bfloat16), None
    # one scale per row (over its 576 numbers), the codes e4m3
    amax = x.abs().amax(dim=(1, 3))
    codes = (x * (448.0 / amax)[:, None, :, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), amax / 448.0


def _table(pages, seed: int, spare: int = 2):
    """Block table [B, most pages] of a shuffled pool, unused entries -1, and the pool's size."""
    total = sum(pages) + spare
    ids = list(range(total))
    random.Random(seed * 16 + 9).shuffle(ids)
    most = max(1, max(pages))
    table, at = [], 0
    for n in pages:
        table.append(ids[at:at + n] + [-1] * (most - n))
        at += n
    return _ints(table), total


def _rope(max_pos: int):
    inv = 10000.0 ** (-2.0 * torch.arange(D_R // 2, device="cuda", dtype=torch.float64) / D_R)
    ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * inv
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"tree": _prepare_tree, "plan": _prepare_plan, "append": _prepare_append,
            "commit": _prepare_commit}[case["op"]](case, seed, gen)


def _prepare_tree(case, seed, gen):
    B, H, cache = case["batch"], case["heads"], case["cache"]
    counts = _shuffled(_spread(case["nodes_lo"], case["nodes_hi"], B), seed, 1)
    prefix = _shuffled(_spread(case["len_lo"], case["len_hi"], B), seed, 2)
    lens = [p + n for p, n in zip(prefix, counts)]
    words = -(-case["nodes_hi"] // 64)
    rng = random.Random(seed * 16 + 3)
    mask = [row for n in counts for row in _ancestor_words(_tree(n, rng), words)]
    table, num_pages = _table([-(-x // PAGE) for x in lens], seed)
    pool, scale = _pool_rows(num_pages, cache, gen)
    starts = _starts(counts)
    N = starts[-1]
    qdt = torch.float32 if cache == "f32" else torch.bfloat16
    # scores of standard deviation near 2 under the 1/sqrt(192) scale
    q = (torch.randn((N, H, D_ROW), generator=gen, device="cuda") * (2.0 / (SCALE * math.sqrt(D_ROW)))).to(qdt)
    s = dict(op="tree", B=B, H=H, N=N, T=max(counts), words=words, cache_kind=cache, q=q, pool=pool, scale=scale,
             num_pages=num_pages, table=table, kv_lens=_ints(lens), row_start=_ints(starts),
             mask=torch.tensor(mask, dtype=torch.int64, device="cuda"),
             o=torch.empty((N, H, D_C), dtype=qdt, device="cuda"),
             lse=torch.empty((N, H), dtype=torch.float32, device="cuda"),
             seq_ids=_ints([b for b, n in enumerate(counts) for _ in range(n)]).long())
    if own:
        import latent_attention_decode_absorbed_b200 as mla
        code = dict(f32=mla.MLA_F32, bf16=mla.MLA_BF16, e4m3=mla.MLA_E4M3)[cache]
        need = mla.mla_decode_tree_workspace_bytes(code, N, H)
        s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


def _prepare_plan(case, seed, gen):
    B, tree = case["batch"], case["tree"]
    counts = _shuffled(_spread(case["nodes_lo"], case["nodes_hi"], B), seed, 1)
    lens = _shuffled(_spread(case["len_lo"], case["len_hi"], B), seed, 2)
    starts = _starts(counts)
    N = starts[-1]
    words = -(-case["nodes_hi"] // 64) if tree else 0
    held = [-(-x // PAGE) for x in lens]
    need = [-(-(x + n) // PAGE) for x, n in zip(lens, counts)]
    most = max(need)
    ids = list(range(sum(need) + 8))
    random.Random(seed * 16 + 9).shuffle(ids)
    table, at = [], 0
    for n in held:
        table.append(ids[at:at + n] + [-1] * (most - n))
        at += n
    free = ids[at:] + [-1] * at
    parents = None
    if tree:
        rng = random.Random(seed * 16 + 3)
        parents = _ints([p for n in counts for p in _tree(n, rng)])
    empty = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(op="plan", B=B, N=N, words=words, num_pages=len(ids), max_pages=most, lens=_ints(lens),
                counts=_ints(counts), parents=parents, held=_ints(held), free=_ints(free),
                free_count=_ints([len(ids) - at]), table=_ints(table), held_out=empty(B), free_count_out=empty(1),
                row_start=empty(B + 1), kv_lens=empty(B), positions=empty(N), slots=empty(N),
                mask=torch.empty((N, words), dtype=torch.int64, device="cuda") if tree else None)


def _prepare_append(case, seed, gen):
    n, cache = case["rows"], case["cache"]
    num_pages = -(-n // PAGE) + 2
    max_pos = 8192
    kv = torch.randn((n, D_ROW), generator=gen, device="cuda").to(
        torch.float32 if cache == "f32" else torch.bfloat16)
    pool = torch.zeros((num_pages, 9, PAGE, 64), dtype=DTYPE[cache], device="cuda")
    scale = torch.zeros((num_pages, PAGE), dtype=torch.float32, device="cuda") if cache == "e4m3" else None
    slots = torch.randperm(num_pages * PAGE, generator=gen, device="cuda")[:n].to(torch.int32)
    positions = torch.randint(0, max_pos, (n,), generator=gen, device="cuda", dtype=torch.int32)
    gain = 1.0 + 0.1 * torch.randn(D_C, generator=gen, device="cuda")
    cos, sin = _rope(max_pos)
    return dict(op="append", n=n, cache_kind=cache, kv=kv, pool=pool, scale=scale, num_pages=num_pages, slots=slots,
                positions=positions, gain=gain, cos=cos, sin=sin, max_pos=max_pos)


def _prepare_commit(case, seed, gen):
    B, n, cache = case["batch"], case["nodes"], case["cache"]
    rng = random.Random(seed * 16 + 3)
    base = _shuffled(_spread(max(1, case["length"] // 2), case["length"], B), seed, 2)
    # accepted paths: the root, then deeper nodes of the breadth-first order
    counts, nodes = [], []
    for _ in range(B):
        c = rng.randint(1, case["count_hi"])
        path = [0] + sorted(rng.sample(range(c, n), c - 1))
        counts.append(c)
        nodes += path + [-1] * (n - c)
    lens = [x + n for x in base]
    table, num_pages = _table([-(-x // PAGE) for x in lens], seed)
    pool, scale = _pool_rows(num_pages, cache, gen)
    return dict(op="commit", B=B, n=n, cache_kind=cache, pool=pool, scale=scale, num_pages=num_pages, table=table,
                kv_lens=_ints(lens), row_start=_ints(_starts([n] * B)), counts=_ints(counts), nodes=_ints(nodes),
                seq_lens=torch.empty(B, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ one pass
def run(s):
    return {"tree": _run_tree, "plan": _run_plan, "append": _run_append, "commit": _run_commit}[s["op"]](s)


def _codes(mla):
    return dict(f32=mla.MLA_F32, bf16=mla.MLA_BF16, e4m3=mla.MLA_E4M3)


def _pool_out(s):
    """The pool as values (8-bit codes as the e4m3 numbers they stand for) and its row scales."""
    if s["scale"] is None:
        return {"pool": s["pool"]}
    return {"pool": s["pool"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def _run_tree(s):
    if own:
        import latent_attention_decode_absorbed_b200 as mla
        code = _codes(mla)[s["cache_kind"]]
        qcode = mla.MLA_F32 if s["cache_kind"] == "f32" else mla.MLA_BF16
        mla.mla_decode_tree(s["q"], qcode, s["pool"], s["scale"], code, s["num_pages"], s["table"],
                            s["table"].shape[1], PAGE, s["kv_lens"], s["row_start"], s["B"], s["N"], s["H"],
                            s["mask"], s["words"], SCALE, s["workspace"], s["o"], qcode, s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    B, H, N, T, kv = s["B"], s["H"], s["N"], s["T"], s["kv_lens"].long()
    start = s["row_start"].long()
    count = start[1:] - start[:-1]
    prefix = kv - count
    # every sequence's rows, padded to the longest table: [B, L, 576]
    pages = s["table"].clamp(min=0).long()
    pool = s["pool"] if s["scale"] is None else s["pool"].view(torch.float8_e4m3fn)
    rows = pool.view(torch.uint8)[pages].view(pool.dtype).permute(0, 1, 3, 2, 4).reshape(B, -1, D_ROW).float()
    if s["scale"] is not None:
        rows = rows * s["scale"][pages].reshape(B, -1, 1)
    L = rows.shape[1]
    t = torch.arange(T, device=rows.device)
    at = (start[:-1, None] + t).clamp(max=N - 1)                      # [B, T]
    j = torch.arange(L, device=rows.device)
    k = (j[None] - prefix[:, None])                                   # [B, L] place in the tree
    word = (k.clamp(min=0) // 64).clamp(max=s["words"] - 1)
    bits = s["mask"][at].gather(2, word[:, None].expand(B, T, L)) >> (k.clamp(min=0) % 64)[:, None] & 1
    seen = ((k < 0)[:, None] | ((k >= 0) & (k < count[:, None]))[:, None] & bits.bool())
    q = s["q"][at].float().reshape(B, T * H, D_ROW)
    z = torch.matmul(q, rows.transpose(1, 2)).mul_(SCALE).view(B, T, H, L)
    z.masked_fill_(~seen[:, :, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    z.sub_(m0).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, T * H, L), rows[..., :D_C]).view(B, T, H, D_C)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m0 + total.log()).squeeze(-1)
    b, n = s["seq_ids"], torch.arange(N, device=rows.device)
    pick = n - start[b]
    return {"o": o[b, pick].to(s["o"].dtype), "lse": lse[b, pick]}


def _run_plan(s):
    if own:
        import latent_attention_decode_absorbed_b200 as mla
        mla.mla_step_plan(s["lens"], s["counts"], s["parents"], s["B"], s["N"], s["words"], s["held"], s["held_out"],
                          s["free"], s["free_count"], s["free_count_out"], s["table"], s["max_pages"], PAGE,
                          s["num_pages"], s["row_start"], s["kv_lens"], None, s["positions"], s["slots"], s["mask"])
        out = {k: s[k] for k in ("held_out", "free_count_out", "table", "row_start", "kv_lens", "positions", "slots")}
        return out if s["mask"] is None else {**out, "mask": s["mask"]}
    B, N, lens, counts = s["B"], s["N"], s["lens"].long(), s["counts"].long()
    start = torch.zeros(B + 1, dtype=torch.int64, device=lens.device)
    start[1:] = counts.cumsum(0)
    kv = lens + counts
    held, need = s["held"].long(), (kv + PAGE - 1) // PAGE
    fresh = (need - held).clamp(min=0)
    first = fresh.cumsum(0) - fresh
    # pages come off the end of the free list, in sequence order
    p = torch.arange(s["max_pages"], device=lens.device)
    new = (p >= held[:, None]) & (p < need[:, None])
    place = s["free_count"].long() - 1 - (first[:, None] + p - held[:, None])
    table = torch.where(new, s["free"][place.clamp(min=0, max=s["num_pages"] - 1)], s["table"])
    n = torch.arange(N, device=lens.device)
    b = torch.searchsorted(start[1:], n, right=True)
    i = n - start[b]
    row = lens[b] + i
    slots = table[b, row // PAGE].long() * PAGE + row % PAGE
    out = dict(held_out=torch.maximum(held, need), free_count_out=s["free_count"] - fresh.sum(), table=table,
               row_start=start, kv_lens=kv, positions=row, slots=slots)
    if s["parents"] is not None:
        # pointer doubling: after r rounds a node knows its ancestors up to 2^r levels above it
        up = torch.where(s["parents"] >= 0, s["parents"].long() + start[b], torch.full_like(n, -1))
        bit = torch.zeros((N, s["words"]), dtype=torch.int64, device=lens.device)
        bit.scatter_(1, (i // 64)[:, None], (torch.ones_like(i) << (i % 64))[:, None])
        depth = (up >= 0).long()
        rounds = max(1, math.ceil(math.log2(64 * s["words"] + 1)))
        for _ in range(rounds):
            has = up >= 0
            at = up.clamp(min=0)
            bit = bit | torch.where(has[:, None], bit[at], torch.zeros_like(bit))
            depth = depth + torch.where(has, depth[at], torch.zeros_like(depth))
            up = torch.where(has, up[at], up)
        out["positions"] = lens[b] + depth
        out["mask"] = bit
    return {k: v if k == "mask" else v.to(torch.int32) for k, v in out.items()}


def _run_append(s):
    if own:
        import latent_attention_decode_absorbed_b200 as mla
        kv_code = mla.MLA_F32 if s["kv"].dtype == torch.float32 else mla.MLA_BF16
        mla.mla_cache_append_slots(s["kv"], kv_code, s["n"], s["slots"], s["positions"], s["gain"], EPS, s["cos"],
                                   s["sin"], s["max_pos"], s["pool"], s["scale"], _codes(mla)[s["cache_kind"]],
                                   s["num_pages"])
        return _pool_out(s)
    x = s["kv"].float()
    c, k = x[:, :D_C], x[:, D_C:].view(-1, D_R // 2, 2)
    c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["gain"]
    at = s["positions"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    k = torch.stack([k[..., 0] * cos - k[..., 1] * sin, k[..., 0] * sin + k[..., 1] * cos], -1).view(-1, D_R)
    row = torch.cat([c, k], 1)
    slot = s["slots"].long()
    if s["scale"] is not None:
        amax = row.abs().amax(1)
        s["scale"].view(-1)[slot] = amax / 448.0
        row = (row * torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))[:, None]).clamp(-448.0, 448.0)
        row = row.to(torch.float8_e4m3fn).view(torch.uint8)
    s["pool"][slot // PAGE, :, slot % PAGE] = row.to(s["pool"].dtype).view(-1, 9, 64)
    return _pool_out(s)


def _run_commit(s):
    if own:
        import latent_attention_decode_absorbed_b200 as mla
        mla.mla_cache_commit(s["kv_lens"], s["row_start"], s["B"], s["B"] * s["n"], s["counts"], s["nodes"],
                             s["table"], s["table"].shape[1], PAGE, s["pool"], s["scale"], _codes(mla)[s["cache_kind"]],
                             s["num_pages"], s["seq_lens"])
        return {**_pool_out(s), "seq_lens": s["seq_lens"]}
    start = s["row_start"].long()
    base = s["kv_lens"].long() - (start[1:] - start[:-1])
    j = torch.arange(s["n"], device=base.device)
    live = j < s["counts"][:, None]
    b = torch.arange(s["B"], device=base.device)[:, None].expand_as(live)[live]
    to = (base[:, None] + j)[live]
    node = s["nodes"][(start[:-1, None] + j)][live].long()
    fro = base[b] + node
    tp, fp = s["table"][b, to // PAGE].long(), s["table"][b, fro // PAGE].long()
    s["pool"][tp, :, to % PAGE] = s["pool"][fp, :, fro % PAGE]
    if s["scale"] is not None:
        s["scale"][tp, to % PAGE] = s["scale"][fp, fro % PAGE]
    return {**_pool_out(s), "seq_lens": (base + s["counts"]).to(torch.int32)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "tree":
        B, H, size = case["batch"], case["heads"], BYTES[case["cache"]]
        qsize = 4 if case["cache"] == "f32" else 2
        nodes = sum(_spread(case["nodes_lo"], case["nodes_hi"], B))
        prefix = sum(_spread(case["len_lo"], case["len_hi"], B))
        row = D_ROW * size + (4 if case["cache"] == "e4m3" else 0)
        moved = (prefix + nodes) * row + nodes * H * (D_ROW * qsize + D_C * qsize + 4)
        pairs = nodes * prefix / B + nodes          # every drafted token sees its prefix and at least itself
        return {"bytes": moved, "flops": 2.0 * H * (D_ROW + D_C) * pairs}
    if case["op"] == "plan":
        nodes = sum(_spread(case["nodes_lo"], case["nodes_hi"], case["batch"]))
        words = -(-case["nodes_hi"] // 64) if case["tree"] else 0
        fresh = nodes // PAGE
        return {"bytes": case["batch"] * 24 + nodes * (8 + (4 + 8 * words if case["tree"] else 0)) + 8 * fresh,
                "flops": 0}
    if case["op"] == "append":
        size, kv = BYTES[case["cache"]], 4 if case["cache"] == "f32" else 2
        return {"bytes": case["rows"] * (D_ROW * (size + kv) + 8 + (4 if case["cache"] == "e4m3" else 0)),
                "flops": 6.0 * D_ROW * case["rows"]}
    rows = case["batch"] * (case["count_hi"] + 1) / 2
    return {"bytes": rows * (2 * (D_ROW * BYTES[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)) + 4)
            + case["batch"] * 20, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "append":
        return _exact_append(s)
    return None          # whole numbers, and rows moved as they are


def _exact_tree(s):
    """Sequence by sequence, drafted token by drafted token."""
    start, lens = s["row_start"].tolist(), s["kv_lens"].tolist()
    table, words = s["table"].tolist(), s["mask"].tolist()
    o = torch.zeros((s["N"], s["H"], D_C), dtype=torch.float64, device="cuda")
    lse = torch.full((s["N"], s["H"]), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(s["B"]):
        n, L = start[b + 1] - start[b], lens[b]
        ids = torch.tensor(table[b][:-(-L // PAGE)], device="cuda")
        x = s["pool"][ids]
        x = (x.view(torch.float8_e4m3fn) if s["scale"] is not None else x).double()
        x = x.permute(0, 2, 1, 3).reshape(-1, D_ROW)
        if s["scale"] is not None:
            x = x * s["scale"][ids].double().reshape(-1, 1)
        x = x[:L]
        for i in range(n):
            r = start[b] + i
            tree = [k for k in range(n) if words[r][k // 64] >> (k % 64) & 1]
            z = s["q"][r].double() @ x.T / math.sqrt(192.0)
            far = torch.ones(L, dtype=torch.bool, device="cuda")
            far[:L - n] = False
            far[[L - n + k for k in tree]] = False
            z[:, far] = float("-inf")
            lse[r] = torch.logsumexp(z, 1)
            o[r] = torch.softmax(z, 1) @ x[:, :D_C]
    return {"o": o, "lse": lse}


def _exact_append(s):
    pool = torch.zeros((s["num_pages"] * PAGE, D_ROW), dtype=torch.float64, device="cuda")
    x = s["kv"].double()
    c = x[:, :D_C]
    c = c / (c.pow(2).sum(1, keepdim=True) / D_C + EPS).sqrt() * s["gain"].double()
    pos = s["positions"].long()
    turn = torch.complex(s["cos"][pos].double(), s["sin"][pos].double())
    k = torch.view_as_real(torch.view_as_complex(x[:, D_C:].reshape(-1, D_R // 2, 2).contiguous()) * turn)
    row = torch.cat([c, k.reshape(-1, D_R)], 1)
    scale = None
    if s["scale"] is not None:
        top = row.abs().amax(1, keepdim=True)
        scale = torch.zeros(s["num_pages"] * PAGE, dtype=torch.float64, device="cuda")
        scale[s["slots"].long()] = top[:, 0] / 448.0
        row = row * 448.0 / top
    pool[s["slots"].long()] = row
    out = {"pool": pool.view(-1, PAGE, 9, 64).permute(0, 2, 1, 3).contiguous()}
    return out if scale is None else {**out, "scale": scale.view(-1, PAGE)}
