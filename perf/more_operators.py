"""What a target's or draft model's pass over a paged cache costs: attention of
a chain or a tree of new tokens over the cached ones, appending their keys and
values to the pages, accepting a path of the tree and moving the accepted
tokens' keys and values together, and branching sequences by sharing pages.

A pool holds one layer's keys or values, [pages, heads, page, dim].  Row b of a
table lists a sequence's pages in order, -1 for none: its position p is slot
p % page of page table[b, p // page].  refs counts the table entries that hold
a page; a page with none is free.

`run` computes each operator either in its plain form (elementary torch
operations, in 32 bits where numbers are computed) or, with `own`, through the
package's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # verifying four drafts of one sequence: latency
        dict(name="attention_b1_t5_l600_bf16", op="attention", batch=1, nodes=5, least=5, heads=32,
             kv=8, dim=128, low=600, high=600, page=16, dtype="bf16", tree=False),
        # single tokens of a ragged batch
        dict(name="attention_b64_t1_l4000_bf16", op="attention", batch=64, nodes=1, least=1,
             heads=32, kv=8, dim=128, low=200, high=4000, page=16, dtype="bf16", tree=False),
        # verifying chains of eight drafts of a ragged batch, some of them trimmed
        dict(name="attention_b64_t9_l8000_bf16", op="attention", batch=64, nodes=9, least=3,
             heads=32, kv=8, dim=128, low=1000, high=8000, page=64, dtype="bf16", tree=False),
        # wide trees, eight query heads to a key head: most arithmetic per key
        dict(name="attention_b16_t64_l12000_f16_tree", op="attention", batch=16, nodes=64, least=40,
             heads=64, kv=8, dim=128, low=4000, high=12000, page=16, dtype="f16", tree=True),
        # two very long caches
        dict(name="attention_b2_t9_l131072_bf16", op="attention", batch=2, nodes=9, least=9,
             heads=64, kv=8, dim=128, low=120001, high=131072, page=128, dtype="bf16", tree=False),
        # a small float32 draft model of odd sizes, an empty cache among its sequences
        dict(name="attention_b5_t13_d80_f32_tree", op="attention", batch=5, nodes=13, least=7,
             heads=6, kv=2, dim=80, low=0, high=1500, page=32, dtype="f32", tree=True),
        # the new tokens of one verified sequence: latency
        dict(name="append_b1_t5_bf16", op="append", batch=1, nodes=5, least=5, kv=8, dim=128,
             low=600, high=600, page=16, dtype="bf16"),
        # a piece of eight prompts
        dict(name="append_b8_t512_bf16", op="append", batch=8, nodes=512, least=301, kv=8, dim=128,
             low=0, high=2000, page=16, dtype="bf16"),
        # one sequence's accepted path, a model of two layers: latency
        dict(name="commit_b1_t8_x4", op="commit", batch=1, nodes=8, least=8, kv=8, dim=128,
             low=600, high=600, page=16, dtype="bf16", layers=2, hit=0.8),
        # a batch of wide trees, a model of four layers
        dict(name="commit_b256_t64_x8", op="commit", batch=256, nodes=64, least=31, kv=8, dim=128,
             low=200, high=1000, page=16, dtype="bf16", layers=4, hit=0.95),
        # four beams of one sequence: latency
        dict(name="branch_b1_w4_x4", op="branch", batch=1, beams=4, kv=8, dim=128, low=600,
             high=600, page=16, dtype="bf16", layers=2, new=1, busy=0.3, pool=4096),
        # eight beams of 64 sequences in a pool of many pages
        dict(name="branch_b64_w8_x8", op="branch", batch=64, beams=8, kv=8, dim=128, low=500,
             high=4000, page=16, dtype="bf16", layers=4, new=5, busy=0.3, pool=40000),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "commit", "branch"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    size = 4 if dtype == "f32" else 2
    page = rng.choice([8, 16, 16, 32, 64, 128, 256])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    if op == "attention":
        heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
        tree = rng.random() < 0.5
        nodes = 1 if rng.random() < 0.2 else _log_int(rng, 2, 128 if tree else 300)
        batch = _log_int(rng, 1, 64)
        # the keys and values of all sequences, and the products with them
        most = min(1.0e9 / (2 * batch * kv * dim * size), 1.8e11 / (4 * batch * heads * nodes * dim),
                   131072)
        high = _log_int(rng, 1, max(1, int(most)))
        return dict(op=op, batch=batch, nodes=nodes, least=rng.randint(0, nodes), heads=heads,
                    kv=kv, dim=dim, low=rng.randint(0, high), high=high, page=page, dtype=dtype,
                    tree=tree)
    if op == "append":
        batch, nodes = _log_int(rng, 1, 256), _log_int(rng, 1, 512)
        nodes = max(1, min(nodes, 8 * 512 // batch))
        high = _log_int(rng, 1, 2000)
        return dict(op=op, batch=batch, nodes=nodes, least=rng.randint(0, nodes), kv=kv, dim=dim,
                    low=rng.randint(0, high), high=high, page=page, dtype=dtype)
    if op == "commit":
        batch = _log_int(rng, 1, 256)
        nodes = _log_int(rng, 1, 128 if batch <= 64 else 64)
        high = _log_int(rng, 1, 1000)
        return dict(op=op, batch=batch, nodes=nodes, least=rng.randint(0, nodes), kv=kv,
                    dim=dim if size * dim <= 256 else 64, low=rng.randint(0, high), high=high,
                    page=page, dtype=dtype, layers=rng.randint(1, 4),
                    hit=round(rng.uniform(0.3, 1.0), 2))
    batch, beams = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8])
    high = _log_int(rng, 1, 2000)
    new = _log_int(rng, 1, 64)
    tail = -(-(48 + new) // page) + 2
    need = batch * (-(-high // page) + 1 + 3 * beams * tail)
    while need * kv * dim * page * size > 1.0e9 and batch > 1:  # a pool's bytes
        batch //= 2
        need = batch * (-(-high // page) + 1 + 3 * beams * tail)
    busy = round(rng.uniform(0.0, 0.6), 2)
    return dict(op=op, batch=batch, beams=beams, kv=kv, dim=dim, low=rng.randint(1, high), high=high,
                page=page, dtype=dtype, layers=rng.randint(1, 4), new=new, busy=busy,
                pool=int(need / (1.0 - busy)) + rng.randint(64, 5000))


def _spread(low, high, count):
    """count numbers spread evenly from high down to low."""
    return [high - (high - low) * i // max(1, count - 1) for i in range(count)]


def _sizes(case):
    """(cached positions, nodes in use) of each sequence."""
    B = case["batch"]
    nodes = _spread(case["least"], case["nodes"], B)
    # paired so that the longest caches do not all have the widest trees
    return _spread(case["low"], case["high"], B), nodes[::2] + nodes[1::2]


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _paged(case, g):
    """(table, lengths, nodes in use, pages of the pool): pages in random order,
    room for every sequence's nodes."""
    lengths, nodes = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in _sizes(case))
    order = torch.randperm(case["batch"], generator=g, device=DEV)
    lengths, nodes = lengths[order], nodes[order]
    page = case["page"]
    held = (lengths + nodes + page - 1) // page
    width = (case["high"] + case["nodes"] + page - 1) // page + 1
    used = torch.arange(width, device=DEV) < held[:, None]
    total = sum(-(-(a + n) // page) for a, n in zip(*_sizes(case)))
    pages = total + 7
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=DEV)
    table[used] = torch.randperm(pages, generator=g, device=DEV)[:total].to(torch.int32)
    return table, lengths, nodes, pages


def _tree(B, T, g):
    """Parents of random trees: node 0 is the root, every other node's parent precedes it."""
    at = torch.arange(T, device=DEV)
    parents = (torch.rand(B, T, generator=g, device=DEV) * at).long().clamp(max=(at - 1).clamp(min=0))
    parents[:, 0] = -1
    return parents.to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    op, dt = case["op"], TYPES[case["dtype"]]
    B, kv, D, page = case["batch"], case["kv"], case["dim"], case["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(dt)

    if op == "branch":
        return _prepare_branch(case, g, normal)
    T = case["nodes"]
    table, lengths, nodes, pages = _paged(case, g)
    s = dict(case=case, table=table, lengths=lengths, nodes=None if case["least"] == T else nodes)
    if op == "attention":
        # a projection's output holds queries, keys and values side by side
        rows = normal(B, T, case["heads"] + 2 * kv, D)
        s.update(q=2.0 * rows, keys=normal(pages, kv, page, D), values=normal(pages, kv, page, D),
                 parents=_tree(B, T, g) if case["tree"] else None)
        s["q"] = s["q"][:, :, :case["heads"]]
    elif op == "append":
        rows = normal(B, T, 3 * kv, D)
        s.update(k=rows[:, :, kv:2 * kv], v=rows[:, :, 2 * kv:], keys=normal(pages, kv, page, D),
                 values=normal(pages, kv, page, D))
    else:
        tokens = torch.randint(0, 8, (B, T), generator=g, device=DEV, dtype=torch.int32)
        parents = _tree(B, T, g)
        # what the target chose after a node: one of its children's tokens in most places
        child = torch.rand(B, T, T, generator=g, device=DEV)
        child = child.masked_fill(parents[:, None, :] != torch.arange(T, device=DEV)[:, None], -1.0)
        best = child.max(dim=-1)
        hit = (torch.rand(B, T, generator=g, device=DEV) < case["hit"]) & (best.values >= 0)
        other = torch.randint(8, 16, (B, T), generator=g, device=DEV, dtype=torch.int32)
        s.update(tokens=tokens, parents=parents,
                 chosen=torch.where(hit, tokens.gather(1, best.indices), other),
                 pools=[normal(pages, kv, page, D) for _ in range(2 * case["layers"])])
    return s


def _prepare_branch(case, g, normal):
    """Sequences whose beams share the prompt's pages and have grown apart, and
    the tables of an older branching that the next one replaces."""
    B, W, page, N = case["batch"], case["beams"], case["page"], case["pool"]
    # pages that other sequences hold
    refs = (torch.rand(N, generator=g, device=DEV) < case["busy"]).to(torch.int32)
    lengths = torch.tensor(_spread(case["low"], case["high"], B), dtype=torch.int32, device=DEV)
    lengths = lengths[torch.randperm(B, generator=g, device=DEV)][:, None]
    width = -(-(case["high"] + 48 + case["new"]) // page) + 1
    prompt = torch.full((B, 1, width), -1, dtype=torch.int32, device=DEV)
    _plain_reserve(prompt, torch.zeros_like(lengths), refs, page, lengths)
    table = torch.full((B, W, width), -1, dtype=torch.int32, device=DEV)
    first = torch.zeros(B, W, dtype=torch.int32, device=DEV)
    used = _plain_fork(prompt, lengths, first, refs, page, table)
    grown = torch.randint(1, 48, (B, W), generator=g, device=DEV, dtype=torch.int32)
    _plain_reserve(table, used, refs, page, grown)
    used = used + grown
    _plain_release(prompt, refs, page)

    def parents():
        return torch.randint(0, W, (B, W), generator=g, device=DEV, dtype=torch.int32)

    branch = torch.full_like(table, -1)
    older = _plain_fork(table, used, parents(), refs, page, branch)
    _plain_reserve(branch, older, refs, page, torch.ones_like(older))
    return dict(case=case, table=table, lengths=used, refs=refs, branch=branch, parents=parents(),
                new=torch.full((B, W), case["new"], dtype=torch.int32, device=DEV),
                pools=[normal(N, case["kv"], page, case["dim"]) for _ in range(2 * case["layers"])])


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _above(parents):
    """[B, T, T]: whether node j is node i or one of its ancestors.  Powers of
    (one + parent) count the ways up; only which are nonzero matters."""
    T = parents.shape[1]
    at = torch.arange(T, device=parents.device)
    step = (parents[:, :, None] == at).float() + torch.eye(T, device=parents.device)
    return torch.linalg.matrix_power(step, max(1, T - 1)) > 0


def _in_use(s, T):
    """[B, T]: whether a node is in use."""
    at = torch.arange(T, device=DEV)
    if s["nodes"] is None:
        return torch.ones(s["lengths"].shape[0], T, dtype=torch.bool, device=DEV)
    return at < s["nodes"][:, None]


def _plain_attention(s):
    q = s["q"].float()
    B, T, H, D = q.shape
    kv = s["keys"].shape[1]
    at = s["table"].clamp(min=0).long()

    def rows(pool):  # [B, kv, positions, D]
        return pool[at].permute(0, 2, 1, 3, 4).reshape(B, kv, -1, D).float()

    keys, values = rows(s["keys"]), rows(s["values"])
    N = keys.shape[2]
    q = q.reshape(B, T, kv, H // kv, D).permute(0, 2, 1, 3, 4).reshape(B, kv, -1, D)
    score = torch.matmul(q, keys.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(D))
    if s["parents"] is None:
        above = torch.ones(T, T, dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    else:
        above = _above(s["parents"])
    use = _in_use(s, T)
    above = above & use[:, None, :]
    node = torch.arange(N, device=DEV) - s["lengths"][:, None]
    seen = above.gather(2, node.clamp(0, T - 1)[:, None, :].expand(B, T, N))
    seen = torch.where((node < 0)[:, None, :], True, seen & (node < T)[:, None, :])
    seen = seen & use[:, :, None] & (s["table"] >= 0).repeat_interleave(N // at.shape[1], 1)[:, None, :]
    seen = seen[:, None, :, None, :].expand(B, kv, T, H // kv, N).reshape(score.shape)
    score = score.masked_fill(~seen, float("-inf"))
    top = score.max(dim=-1, keepdim=True).values
    top = top.masked_fill(top == float("-inf"), 0.0)
    weight = (score - top).exp()
    total = weight.sum(dim=-1, keepdim=True)
    values = values.masked_fill((node >= T)[:, None, :, None], 0.0)
    out = torch.matmul(weight, values) / total.masked_fill(total == 0, 1.0)
    lse = (top + total.log()).squeeze(-1)

    def back(x):
        x = x.reshape((B, kv, T, H // kv) + x.shape[3:])
        return x.transpose(1, 2).reshape((B, T, H) + x.shape[4:])

    return back(out).to(s["q"].dtype), back(lse)


def _slots(s, position, page):
    """(page, slot) of positions [B, n]."""
    at = s["table"].gather(1, position // page).long()
    return at, position % page


def _plain_append(s):
    T, page = s["k"].shape[1], s["case"]["page"]
    use = _in_use(s, T)
    position = s["lengths"].long()[:, None] + torch.arange(T, device=DEV)
    at, slot = _slots(s, torch.where(use, position, 0), page)
    at, slot = at[use], slot[use]

    def one(pool, new):
        pool[at, :, slot] = new[use]
        return pool

    return one(s["keys"], s["k"]), one(s["values"], s["v"])


def _plain_accept(s):
    parents, tokens, chosen = s["parents"].long(), s["tokens"], s["chosen"]
    B, T = parents.shape
    at = torch.arange(T, device=DEV)
    use = _in_use(s, T)
    up = parents.clamp(min=0)
    good = (tokens == chosen.gather(1, up)) & (parents >= 0) & use
    twin = (parents[:, :, None] == parents[:, None, :]) & good[:, None, :] & (at[:, None] > at)
    good = good & ~twin.any(dim=-1)
    good[:, 0] = use[:, 0]
    on = torch.matmul(_above(s["parents"]).float(), (~good).float()[:, :, None])[:, :, 0] == 0
    count = on.sum(dim=1)
    path = torch.where(on, at, T).sort(dim=1).values
    live = at < count[:, None]
    here = path.clamp(max=T - 1)
    after = torch.cat([here[:, 1:], here[:, :1]], dim=1)
    last = at == count[:, None] - 1
    token = torch.where(last, chosen.gather(1, here), tokens.gather(1, after))
    return (torch.where(live, path, -1).to(torch.int32), count.to(torch.int32),
            torch.where(live, token, -1).to(torch.int32))


def _plain_commit(s):
    path, count, tokens = _plain_accept(s)
    T, page = path.shape[1], s["case"]["page"]
    step = torch.arange(T, device=DEV)
    use = step < count[:, None]
    start = s["lengths"].long()[:, None]
    to = _slots(s, torch.where(use, start + step, 0), page)
    of = _slots(s, torch.where(use, start + path, 0), page)
    to, of = [x[use] for x in to], [x[use] for x in of]

    def one(pool):
        pool[to[0], :, to[1]] = pool[of[0], :, of[1]]
        return pool

    return path, count, tokens, s["lengths"] + count, [one(pool) for pool in s["pools"]]


def _plain_release(table, refs, page):
    held = table >= 0
    refs.scatter_add_(0, table.clamp(min=0).flatten().long(), -held.flatten().to(torch.int32))
    table.fill_(-1)


def _plain_fork(table, lengths, parents, refs, page, out):
    at = parents.long()
    rows = table.gather(1, at[:, :, None].expand(-1, -1, table.shape[2]))
    used = lengths.gather(1, at)
    held = torch.arange(table.shape[2], device=DEV) < ((used + page - 1) // page)[:, :, None]
    out.copy_(torch.where(held, rows, -1))
    held = out >= 0
    refs.scatter_add_(0, out.clamp(min=0).flatten().long(), held.flatten().to(torch.int32))
    return used


def _plain_reserve(table, lengths, refs, page, new):
    P = table.shape[-1]
    tab, L, new = table.view(-1, P), lengths.reshape(-1, 1).long(), new.reshape(-1, 1).long()
    at = torch.arange(P, device=DEV)
    need = (at >= L // page) & (at < (L + new + page - 1) // page) & (new > 0)
    have = need & (tab >= 0)
    held = tab.clamp(min=0).long()
    shared = have & (refs[held] > 1)
    # a shared page whose every holder is here stays with the first of them
    holders = torch.zeros_like(refs).scatter_add_(0, held.flatten(), shared.flatten().to(torch.int32))
    place = torch.arange(tab.numel(), device=DEV).view(tab.shape)
    first = torch.full(refs.shape, tab.numel(), dtype=torch.long, device=DEV)
    first.scatter_reduce_(0, held.flatten(), torch.where(shared, place, tab.numel()).flatten(), "amin")
    stays = shared & (holders[held] == refs[held]) & (first[held] == place)
    fresh = need & (~have | (shared & ~stays))
    rank = fresh.flatten().long().cumsum(0).view(tab.shape) - 1
    free = refs <= 0
    missing = (fresh.sum() - free.sum()).clamp(min=0).to(torch.int32)
    fresh = fresh & (missing == 0)
    order = torch.sort((~free).to(torch.uint8), stable=True).indices
    taken = order[rank.clamp(0, refs.numel() - 1)]
    moved = fresh & have & (at == L // page) & (L % page > 0)
    copies = torch.stack([torch.where(moved, tab, 0).sum(1), torch.where(moved, taken, 0).sum(1),
                          torch.where(moved, L % page, 0).sum(1)], dim=1)
    copies = torch.where(moved.any(dim=1)[:, None], copies, torch.tensor([-1, -1, 0], device=DEV))
    refs.scatter_add_(0, held.flatten(), -(fresh & have).flatten().to(torch.int32))
    refs.scatter_add_(0, taken.flatten(), fresh.flatten().to(torch.int32))
    tab.copy_(torch.where(fresh, taken.to(torch.int32), tab))
    return copies.to(torch.int32), missing.reshape(1)


def _plain_copy(pools, copies, page):
    copies = copies[copies[:, 0] >= 0].long()
    keep = (torch.arange(page, device=DEV) < copies[:, 2:])[:, None, :, None]

    def one(pool):
        pool[copies[:, 1]] = torch.where(keep, pool[copies[:, 0]], pool[copies[:, 1]])
        return pool

    return [one(pool) for pool in pools]


def _plain_branch(s):
    page = s["case"]["page"]
    _plain_release(s["branch"], s["refs"], page)
    used = _plain_fork(s["table"], s["lengths"], s["parents"], s["refs"], page, s["branch"])
    copies, missing = _plain_reserve(s["branch"], used, s["refs"], page, s["new"])
    pools = _plain_copy(s["pools"], copies, page)
    return s["branch"], used, s["refs"], copies, missing, pools


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import draft_token_verification_vocab_amd as sv
        if op == "attention":
            return sv.tree_attention(state["q"], state["keys"], state["values"], state["table"],
                                     state["lengths"], state["parents"], num_nodes=state["nodes"],
                                     lse=True)
        if op == "append":
            return sv.cache_append(state["k"], state["v"], state["keys"], state["values"],
                                   state["table"], state["lengths"], num_nodes=state["nodes"])
        if op == "commit":
            r = sv.tree_accept(state["parents"], state["tokens"], state["chosen"],
                               num_nodes=state["nodes"])
            lengths = sv.cache_keep(state["pools"], state["table"], state["lengths"], r["path"],
                                    r["count"])
            return r["path"], r["count"], r["tokens"], lengths, state["pools"]
        sv.pages_release(state["branch"], state["refs"], c["page"])
        used = sv.pages_fork(state["table"], state["lengths"], state["parents"], state["refs"],
                             c["page"], out=state["branch"])
        r = sv.pages_reserve(state["branch"], used, state["refs"], c["page"], state["new"])
        sv.pages_copy(state["pools"], r["copies"])
        return state["branch"], used, state["refs"], r["copies"], r["missing"], state["pools"]
    if op == "attention":
        return _plain_attention(state)
    if op == "append":
        return _plain_append(state)
    if op == "commit":
        return _plain_commit(state)
    return _plain_branch(state)


def work(case):
    """Each input read once, each output written once.  Attention: two products
    of each query with the keys that it sees (of a tree's nodes it sees about
    ln T + 1 above it).  Of moved positions and copied pages the half, as an
    expectation; of tables and reference counts the entries in use."""
    op, size = case["op"], 4 if case["dtype"] == "f32" else 2
    row = case["kv"] * case["dim"] * size
    if op == "branch":
        B, W, page = case["batch"], case["beams"], case["page"]
        held = sum(-(-(a + 24) // page) for a in _spread(case["low"], case["high"], B)) * W
        copied = 2 * case["layers"] * B * W * row * page // 2
        return dict(bytes=2 * copied + 4 * (5 * held + case["pool"]), flops=0)
    pairs = list(zip(*_sizes(case)))
    if op == "append":
        return dict(bytes=4 * row * sum(n for _, n in pairs), flops=0)
    if op == "commit":
        deep = 1.0 / max(0.05, 1.0 - case["hit"])
        moved = sum(min(math.log(n + 1.0), deep) for _, n in pairs)
        return dict(bytes=int(2 * 2 * case["layers"] * row * moved)
                    + 20 * case["batch"] * case["nodes"], flops=0)
    seen = (lambda n: n * (math.log(n + 1.0) + 1.0)) if case["tree"] else (lambda n: n * (n + 1) / 2)
    live = [(a, n) for a, n in pairs if n > 0]
    nodes, heads = case["batch"] * case["nodes"], case["heads"]
    return dict(bytes=2 * row * sum(a + n for a, n in live)
                + heads * case["dim"] * size * (sum(n for _, n in live) + nodes) + 4 * heads * nodes,
                flops=int(4 * case["dim"] * heads * sum(n * a + seen(n) for a, n in live)))


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    """Attention, sequence by sequence.  The other operators move what they are
    given and compute no numbers."""
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    B, T, H, D = s["q"].shape
    kv, page = case["kv"], case["page"]
    out = torch.zeros(B, T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, H), float("-inf"), dtype=torch.float64, device=DEV)
    parents = None if s["parents"] is None else s["parents"].tolist()
    nodes = [T] * B if s["nodes"] is None else s["nodes"].tolist()
    for b, (L, n) in enumerate(zip(s["lengths"].tolist(), nodes)):
        if n == 0:
            continue
        see = np.zeros((n, L + n), dtype=bool)
        see[:, :L] = True
        for i in range(n):
            j = i
            while j >= 0:
                see[i, L + j] = True
                j = j - 1 if parents is None else parents[b][j]
        see = torch.from_numpy(see).to(DEV)
        pages = s["table"][b, :-(-(L + n) // page)].long()
        for h in range(kv):
            k, v = (pool[pages, h].reshape(-1, D)[:L + n].double() for pool in (s["keys"], s["values"]))
            for m in range(h * (H // kv), (h + 1) * (H // kv)):
                z = (s["q"][b, :n, m].double() @ k.t()) / math.sqrt(D)
                z = z.masked_fill(~see, float("-inf"))
                lse[b, :n, m] = torch.logsumexp(z, dim=-1)
                out[b, :n, m] = torch.softmax(z, dim=-1) @ v
    return out, lse
