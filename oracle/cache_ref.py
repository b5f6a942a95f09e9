"""Plain 64-bit definitions of the paged-cache calls, sequence by sequence:
attention of a chain or a tree of new tokens over paged keys and values,
appending, accepting a path, keeping it, and the pages' bookkeeping.  Test
infrastructure only."""
import numpy as np
import torch


def span(length, nodes, width, page):
    """(cached, positions) of a sequence as far as its table row reaches."""
    room = width * page
    cached = min(max(int(length), 0), room)
    return cached, 0 if nodes == 0 else min(cached + nodes, room)


def held(table_row, p, page, num_pages):
    """The page that holds position p, or None."""
    e = int(table_row[p // page])
    return e if 0 <= e < num_pages else None


def ancestors(parents, nodes):
    """[nodes][nodes] bool: j is i or above it.  parents None: a chain."""
    see = np.zeros((nodes, nodes), dtype=bool)
    for i in range(nodes):
        see[i, i] = True
        up = i - 1 if parents is None else int(parents[i])
        if 0 <= up < i:
            see[i] |= see[up]
    return see


def in_use(num_nodes, b, T):
    return T if num_nodes is None else min(max(int(num_nodes[b]), 0), T)


def tree_attention(q, keys, values, table, lengths, parents=None, num_nodes=None, scale=None):
    """float64 (out [B, T, H, D], lse [B, T, H]) and what bounds an evaluation in
    fewer bits: mass [B, T, H, D], the weights' sum of |v|; size [B, T, H], the largest
    sum of |scale q k| of a visible key; seen [B, T, H], the visible keys; high [B, H, D],
    the largest |v|."""
    B, T, H, D = q.shape
    N, kv, page, _ = keys.shape
    G = H // kv
    scale = D ** -0.5 if scale is None else scale
    q = q.double()
    out = torch.zeros(B, T, H, D, dtype=torch.float64)
    mass = torch.zeros_like(out)
    high = torch.zeros(B, H, D, dtype=torch.float64)
    lse = torch.full((B, T, H), float("-inf"), dtype=torch.float64)
    size, seen = torch.zeros(B, T, H, dtype=torch.float64), torch.zeros(B, T, H)
    for b in range(B):
        n = in_use(num_nodes, b, T)
        cached, total = span(lengths[b], n, table.shape[1], page)
        above = ancestors(None if parents is None else parents[b].tolist(), n)
        at = [(p, held(table[b], p, page, N)) for p in range(total)]
        at = [(p, e) for p, e in at if e is not None]
        if not at or n == 0:
            continue
        pages = torch.tensor([e for _, e in at])
        slots = torch.tensor([p % page for p, _ in at])
        where = np.array([p for p, _ in at])
        see = (where < cached) | above[:, np.maximum(where - cached, 0)]
        see = torch.from_numpy(see)
        rows = see.repeat_interleave(G, 0)  # a head's rows, node by node
        for h in range(kv):
            k, v = keys[pages, h, slots].double(), values[pages, h, slots].double()
            heads = slice(h * G, (h + 1) * G)
            x = q[b, :n, heads].reshape(n * G, D)
            z = (scale * (x @ k.T)).masked_fill(~rows, float("-inf"))
            total = torch.logsumexp(z, 1)
            w = torch.exp(z - total[:, None])
            w[(total == float("-inf"))] = 0.0
            # a value that is not finite reaches the rows that see it
            odd = ~torch.isfinite(v)
            o = w @ v.masked_fill(odd, 0.0)
            for p in odd.any(1).nonzero()[:, 0].tolist():
                o[rows[:, p]] += torch.where(odd[p], v[p], 0.0)
            u = v.masked_fill(odd, 0.0).abs()
            big = scale * (x.abs() @ k.abs().T)
            lse[b, :n, heads] = total.view(n, G)
            out[b, :n, heads] = o.view(n, G, D)
            mass[b, :n, heads] = (w @ u).view(n, G, D)
            size[b, :n, heads] = big.masked_fill(~rows, 0.0).amax(1).view(n, G)
            seen[b, :n, heads] = rows.sum(1).view(n, G).float()
            high[b, heads] = u.amax(0)
    return out, lse, mass, size, seen, high


def cache_append(k, v, keys, values, table, lengths, num_nodes=None):
    """keys and values with the nodes written, as copies."""
    keys, values = keys.clone(), values.clone()
    N, _, page, _ = keys.shape
    T = k.shape[1]
    for b in range(k.shape[0]):
        n = in_use(num_nodes, b, T)
        cached, total = span(lengths[b], n, table.shape[1], page)
        for j in range(total - cached):
            e = held(table[b], cached + j, page, N)
            if e is not None:
                keys[e, :, (cached + j) % page] = k[b, j]
                values[e, :, (cached + j) % page] = v[b, j]
    return keys, values


def tree_accept(parents, tokens, chosen, num_nodes=None):
    """numpy (path, count, emitted)."""
    B, T = tokens.shape
    path, emitted = np.full((B, T), -1), np.full((B, T), -1)
    count = np.zeros(B, dtype=int)
    for b in range(B):
        n = in_use(num_nodes, b, T)
        at = 0 if n else None
        while at is not None:
            path[b, count[b]] = at
            emitted[b, count[b]] = chosen[b, at]
            count[b] += 1
            kids = [c for c in range(at + 1, n)
                    if parents[b, c] == at and tokens[b, c] == chosen[b, at]]
            at = kids[0] if kids else None
    return path, count, emitted


def cache_keep(pools, table, lengths, path, count):
    """(copies of the pools, new lengths)."""
    old, pools = pools, [p.clone() for p in pools]
    N, _, page, _ = pools[0].shape
    B, T = path.shape
    room = table.shape[1] * page
    new = []
    for b in range(B):
        length = min(max(int(lengths[b]), 0), room)
        n = min(max(int(count[b]), 0), T)
        for i in range(n):
            if not (int(path[b, i - 1]) if i else -1) < int(path[b, i]) < T:
                n = i
                break
        for i in range(n):
            p, t = length + int(path[b, i]), length + i
            if p >= room:
                continue
            e, f = held(table[b], p, page, N), held(table[b], t, page, N)
            if e is None or f is None:
                continue
            for src, dst in zip(old, pools):
                dst[f, :, t % page] = src[e, :, p % page]
        new.append(min(length + n, room))
    return pools, new


def pages_fork(table, lengths, parents, refs, page):
    """numpy (out, out_lengths, refs)."""
    B, W, P = table.shape
    n, refs = parents.shape[1], refs.copy()
    out, new = np.full((B, n, P), -1), np.zeros((B, n), dtype=int)
    for b in range(B):
        for i in range(n):
            w = parents[b, i]
            if not 0 <= w < W:
                continue
            new[b, i] = lengths[b, w]
            use = -(-min(max(int(lengths[b, w]), 0), P * page) // page)
            for k, e in enumerate(table[b, w, :use]):
                if 0 <= e < len(refs):
                    out[b, i, k] = e
                    refs[e] += 1
    return out, new, refs


def pages_release(table, refs, page, lengths=None):
    """numpy (table [rows, P], refs)."""
    table, refs = table.copy(), refs.copy()
    for r, row in enumerate(table):
        use = 0 if lengths is None else min(max(int(lengths[r]), 0), row.size * page)
        for k in range(-(-use // page), row.size):
            if 0 <= row[k] < len(refs) and refs[row[k]] > 0:
                refs[row[k]] -= 1
            row[k] = -1
    return table, refs


def pages_reserve(table, lengths, refs, page, new):
    """numpy (table [rows, P], refs, copies [rows, 3], missing)."""
    start, before = table.copy(), refs.copy()
    table, refs = table.copy(), refs.copy()
    R, P = table.shape
    none = np.tile(np.array([-1, -1, 0]), (R, 1))
    copies = none.copy()
    free = [e for e in range(len(refs)) if refs[e] <= 0]
    wanted = []
    for r in range(R):
        length, more = min(max(int(lengths[r]), 0), P * page), max(int(new[r]), 0)
        if more and int(lengths[r]) + more > P * page:
            return start, before, none, -1
        wanted += [(r, k) for k in range(length // page, -(-(length + more) // page) if more else 0)]
    shared = [(r, k) for r, k in wanted if 0 <= table[r, k] < len(refs) and refs[table[r, k]] > 1]
    holders = {}
    for r, k in shared:
        holders.setdefault(int(table[r, k]), []).append((r, k))
    stay = {who[0] for e, who in holders.items() if len(who) >= refs[e]}
    take = [(r, k) for r, k in wanted
            if not 0 <= table[r, k] < len(refs) or ((r, k) in set(shared) and (r, k) not in stay)]
    if len(take) > len(free):
        return start, before, none, len(take) - len(free)
    for (r, k), page_new in zip(take, free):
        old = int(table[r, k])
        if 0 <= old < len(refs):
            refs[old] -= 1
            if k == int(lengths[r]) // page and int(lengths[r]) % page:
                copies[r] = old, page_new, int(lengths[r]) % page
        table[r, k] = page_new
        refs[page_new] = 1
    return table, refs, copies, 0


def pages_copy(pools, copies):
    old, pools = pools, [p.clone() for p in pools]
    for e, f, n in copies.tolist():
        if 0 <= e < pools[0].shape[0] and 0 <= f < pools[0].shape[0]:
            for src, dst in zip(old, pools):
                dst[f, :, :max(n, 0)] = src[e, :, :max(n, 0)]
    return pools
