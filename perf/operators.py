"""What is timed of the speculative-decoding operators over the paged latent cache.

Four operators of one serving step: ``mla_block_table_update`` (block tables and slot maps
from request lengths), ``mla_tree_mask`` (visibility bits and positions of drafted trees),
``mla_tree_attention`` (every drafted token of a request attends to its cached context and its
own ancestors, absorbed-weight form) and ``mla_tree_commit`` (accepted tokens' cache rows moved
to consecutive positions).  A case is a dict of plain values; ``run`` makes one pass over a
prepared state, in elementary torch operations or, where ``own`` is true, with the package's
kernels; ``exact`` computes the same outputs apart from both, in 64 bits.
"""
import random
import zlib

import numpy as np
import torch

own = False

E, DV = 576, 512            # cache row: 512 latent + 64 rope values; values are the first 512
SM_SCALE = 192 ** -0.5      # the head dim before absorption is 128 + 64

_mla = None


def _pkg():
    global _mla
    if _mla is None:
        import chunked_prefill_attention_ragged_gb300 as m
        _mla = m
    return _mla


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # One request verifying nothing yet: its next token over a short context, 16 heads (the
        # heads of one GPU of eight): the latency of a call.
        {"name": "attn_1x1_over_700_h16", "op": "attention", "nodes_lo": 1, "nodes": 1, "batch": 1, "ctx_lo": 700, "ctx": 700,
         "heads": 16, "block": 64, "tree": False, "cap": 0.0},
        # Single tokens of many requests, 16 heads: bound by reading the cache.
        {"name": "attn_64x1_over_4096_h16", "op": "attention", "nodes_lo": 1, "nodes": 1, "batch": 64, "ctx_lo": 4096, "ctx": 4096,
         "heads": 16, "block": 64, "tree": False, "cap": 0.0},
        # Single tokens with every head on one GPU, ragged contexts.
        {"name": "attn_32x1_ragged_h128", "op": "attention", "nodes_lo": 1, "nodes": 1, "batch": 32, "ctx_lo": 129, "ctx": 16001,
         "heads": 128, "block": 64, "tree": False, "cap": 0.0},
        # One long request, a small tree of drafts: split over the whole GPU.
        {"name": "attn_1x5_over_65537_h128", "op": "attention", "nodes_lo": 5, "nodes": 5, "batch": 1, "ctx_lo": 65537, "ctx": 65537,
         "heads": 128, "block": 64, "tree": True, "cap": 0.0},
        # Ragged trees over small pages, odd counts, capped logits.
        {"name": "attn_9x37_ragged_h16_page16", "op": "attention", "nodes_lo": 3, "nodes": 37, "batch": 9, "ctx_lo": 1, "ctx": 5001,
         "heads": 16, "block": 16, "tree": True, "cap": 30.0},
        # The batch that prefill runs at 128 heads, verifying 16 drafts per request: compute bound.
        {"name": "attn_32x16_over_8192_h128", "op": "attention", "nodes_lo": 16, "nodes": 16, "batch": 32, "ctx_lo": 8192, "ctx": 8192,
         "heads": 128, "block": 64, "tree": True, "cap": 0.0},
        # Block tables of a decode batch in which every request brings a tree of drafts.
        {"name": "tables_100x17_page16", "op": "tables", "batch": 100, "seq_lo": 1, "seq": 9000, "new_lo": 3, "new": 17, "block": 16},
        # Prompts admitted together: every block is new and a slot map of half a million tokens.
        {"name": "tables_128_prompts", "op": "tables", "batch": 128, "seq_lo": 0, "seq": 0, "new_lo": 100, "new": 8192, "block": 64},
        # Trees of one request, and of a large batch.
        {"name": "mask_1x8", "op": "mask", "batch": 1, "nodes_lo": 8, "nodes": 8, "ctx_lo": 1000, "ctx": 1000},
        {"name": "mask_256x61", "op": "mask", "batch": 256, "nodes_lo": 1, "nodes": 100, "ctx_lo": 1, "ctx": 9000},
        # Accepted drafts of a batch, all layers of the cache.
        {"name": "commit_3x1_layer", "op": "commit", "batch": 3, "nodes": 16, "accept_lo": 2, "accept": 5, "layers": 1, "block": 64},
        {"name": "commit_64x60_layers", "op": "commit", "batch": 64, "nodes": 33, "accept_lo": 1, "accept": 9, "layers": 60,
         "block": 64},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "tables", "mask", "commit"])
    block = rng.choice([16, 32, 64, 64, 128, 24])
    if op == "attention":
        heads = rng.choice([1, 5, 8, 16, 16, 32, 48, 64, 128, 128])
        batch = _log(rng, 1, 96)
        tree = rng.random() < 0.6
        n1 = _log(rng, 1, 80) if tree or rng.random() < 0.3 else 1
        n0 = rng.randint(1, n1)
        c1 = _log(rng, 1, 60000)
        c0 = rng.randint(max(1, c1 // 20), c1)
        # no dearer than the largest listed case, in operations and in cached tokens
        while batch > 1 and (batch * n1 * heads * (c1 + n1) > 32 * 16 * 128 * 8192 or batch * c1 > 400000):
            batch = max(1, batch // 2)
        while n1 > 1 and n1 * heads * (c1 + n1) * batch > 32 * 16 * 128 * 8192:
            n1, n0 = max(1, n1 // 2), 1
        return {"op": op, "nodes_lo": n0, "nodes": n1, "batch": batch, "ctx_lo": c0, "ctx": c1, "heads": heads, "block": block,
                "tree": tree, "cap": rng.choice([0.0, 0.0, 30.0])}
    if op == "tables":
        s1 = rng.choice([0, _log(rng, 1, 9000)])
        n1 = _log(rng, 1, 4000)
        batch = max(1, min(_log(rng, 1, 700), 500000 // n1))
        return {"op": op, "batch": batch, "seq_lo": rng.randint(0, s1), "seq": s1, "new_lo": rng.randint(0, n1), "new": n1,
                "block": block}
    if op == "mask":
        n1 = _log(rng, 1, 130)
        return {"op": op, "batch": _log(rng, 1, 256), "nodes_lo": rng.randint(1, n1), "nodes": n1, "ctx_lo": 0, "ctx": _log(rng, 1, 9000)}
    nodes = _log(rng, 2, 64)
    return {"op": op, "batch": _log(rng, 1, 64), "nodes": nodes, "accept_lo": 0, "accept": min(nodes, _log(rng, 1, 12)),
            "layers": _log(rng, 1, 60), "block": block}


def work(case):
    b = case["batch"]
    if case["op"] == "attention":
        n, ctx = _mean(case, "nodes"), _mean(case, "ctx")
        t = b * n * case["heads"]
        mask = b * n * 8 if case["tree"] else 0
        return {"bytes": int(b * (ctx + n) * (E * 2 + 4 / case["block"]) + t * (E * 2 + DV * 2 + 4) + mask + 8 * b),
                "flops": int(2 * t * (ctx + 1) * (E + DV))}
    if case["op"] == "tables":
        # two calls: reserve and roll back
        seq, new = _mean(case, "seq"), _mean(case, "new")
        moved = b * new / case["block"]
        return {"bytes": int(2 * (28 * b + 8 * moved) + b * new * 8 + 4 * moved), "flops": 0}
    if case["op"] == "mask":
        t = b * _mean(case, "nodes")
        return {"bytes": int(t * (4 + 8 * _words(case["nodes"]) + 4) + 8 * b), "flops": 0}
    moved = max(b * (_mean(case, "accept") - 0.5), 0.5) * case["layers"]
    return {"bytes": int(2 * moved * E * 2 + 4 * b * (1 + _mean(case, "accept"))), "flops": 0}


def _mean(case, what):
    return (case[what + "_lo"] + case[what]) / 2


def _words(nodes):
    return (nodes + 63) // 64


# ------------------------------------------------------------------------------ the inputs
def _lengths(rng, case, what):
    """One length per request, from case[what + "_lo"] to case[what], the two ends among them."""
    lo, hi, batch = case[what + "_lo"], case[what], case["batch"]
    out = rng.integers(lo, hi + 1, size=batch)
    out[0] = hi
    if batch > 1:
        out[-1] = lo
    return out.astype(np.int64)


def _indptr(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _trees(rng, nodes):
    """Parents of every request's nodes (-1: a child of the context), each before its child;
    deep and bushy trees both occur, as drafting a few best continuations makes them."""
    out = []
    for n in nodes:
        reach = int(rng.integers(1, 9))
        p = np.array([int(rng.integers(max(-1, i - reach), i)) for i in range(int(n))], dtype=np.int32)
        p[:1] = -1
        out.append(p)
    return np.concatenate(out) if out else np.zeros(0, np.int32)


def _ancestors(parents, qo):
    """Host visibility of every node: its own bit and its ancestors', int64 [T, words]."""
    words = _words(int(np.diff(qo).max(initial=1)))
    bits = np.zeros((len(parents), words), dtype=np.uint64)
    depth = np.zeros(len(parents), dtype=np.int64)
    for r in range(len(qo) - 1):
        for t in range(int(qo[r]), int(qo[r + 1])):
            i, p = t - int(qo[r]), int(parents[t])
            if p >= 0:
                bits[t] = bits[qo[r] + p]
                depth[t] = depth[qo[r] + p] + 1
            bits[t, i >> 6] |= np.uint64(1) << np.uint64(i & 63)
    return bits.view(np.int64), depth


def _paged(rng, lens, block, spare=3):
    """A block table of random distinct blocks for requests of these lengths."""
    need = -(-lens // block)
    total = int(need.sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(lens), max(1, int(need.max()))), -1, dtype=np.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = perm[at:at + k]
        at += int(k)
    return table, total, perm[at:]


def _host(case, seed):
    """Lengths, tables, trees and paths: everything but the large tensors, on the host."""
    rng = np.random.default_rng([seed, 77])
    # lengths belong to the case, so that every seed's outputs have the same shapes
    sizes = np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    h = {"op": case["op"]}
    if case["op"] == "attention":
        nodes, ctx = _lengths(sizes, case, "nodes"), _lengths(sizes, case, "ctx")
        h["qo"], h["kv"] = _indptr(nodes), (nodes + ctx).astype(np.int32)
        h["table"], h["blocks"], _ = _paged(rng, nodes + ctx, case["block"])
        if case["tree"]:
            h["mask"], _ = _ancestors(_trees(rng, nodes), h["qo"])
    elif case["op"] == "tables":
        seq, new = _lengths(sizes, case, "seq"), _lengths(sizes, case, "new")
        bs = case["block"]
        width = int((-(-(seq + new) // bs)).max(initial=1)) + 2
        grow = int((-(-(seq + new) // bs) - -(-seq // bs)).sum())
        table, total, free = _paged(rng, seq, bs, spare=grow + 11)
        h["table"] = np.full((case["batch"], width), -1, dtype=np.int32)
        h["table"][:, :table.shape[1]] = table[:, :width]
        h["held"] = (-(-seq // bs)).astype(np.int32)
        h["free"] = np.full(total, -1, dtype=np.int32)
        h["free"][:len(free)] = free
        h["count"] = np.array([len(free)], dtype=np.int32)
        h["seq"], h["new"] = seq.astype(np.int32), new.astype(np.int32)
        h["tokens"] = int(new.sum()) + 5      # the slot map of a padded batch
    elif case["op"] == "mask":
        nodes, ctx = _lengths(sizes, case, "nodes"), _lengths(sizes, case, "ctx")
        h["qo"], h["kv"] = _indptr(nodes), (nodes + ctx).astype(np.int32)
        h["parents"] = _trees(rng, nodes)
        h["words"] = _words(int(nodes.max()))
    else:
        acc = _lengths(sizes, case, "accept")
        width = max(1, int(acc.max()))
        paths = np.full((case["batch"], width), -1, dtype=np.int32)
        for r, k in enumerate(acc):
            # increasing nodes; the first may stay, the others come from beyond the kept rows
            k = min(int(k), case["nodes"])
            room = np.arange(k, case["nodes"])
            stay = max(k - len(room), 1 if k and rng.random() < 0.5 else 0)
            paths[r, :stay] = np.arange(stay)
            paths[r, stay:k] = np.sort(rng.permutation(room)[:k - stay])
            acc[r] = k
        seq = sizes.integers(0, 300, size=case["batch"])
        h["table"], h["blocks"], _ = _paged(rng, seq + case["nodes"], case["block"])
        h["seq"], h["paths"], h["acc"] = seq.astype(np.int32), paths, acc.astype(np.int32)
    return h


def _big(case, h, seed):
    """The large tensors, bf16 N(0, 1), on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    bf = dict(dtype=torch.bfloat16, device="cuda", generator=g)
    if case["op"] == "attention":
        return {"cache": torch.randn((h["blocks"], case["block"], E), **bf),
                "q": torch.randn((int(h["qo"][-1]), case["heads"], E), **bf)}
    if case["op"] == "commit":
        return {"cache": torch.randn((case["layers"], h["blocks"], case["block"], E), **bf)}
    return {}


def prepare(case, seed):
    h = _host(case, seed)
    s = {"case": case, "host": h}
    for k, v in h.items():
        if isinstance(v, np.ndarray):
            s[k] = torch.from_numpy(v.copy()).to("cuda")
    s.update(_big(case, h, seed))
    if case["op"] == "tables":
        s["zero"] = torch.zeros_like(s["new"])
    return s


# ------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_attention(s):
    c = s["case"]
    return _pkg().mla_tree_attention(s["q"], s["cache"], s["table"], s["qo"], s["kv"], s.get("mask"),
                                     sm_scale=SM_SCALE, logits_soft_cap=c["cap"])


def _own_tables(s):
    m, bs, tokens = _pkg(), s["case"]["block"], s["host"]["tokens"]
    # a step reserves room for its new tokens ...
    out = m.mla_block_table_update(s["seq"], s["new"], s["table"], s["held"], s["free"], s["count"], bs, tokens)
    # ... and, its drafts refused, gives the blocks back
    m.mla_block_table_update(s["seq"], s["zero"], s["table"], s["held"], s["free"], s["count"], bs, 0)
    return list(out) + [s["table"], s["held"], s["free"], s["count"]]


def _own_mask(s):
    return _pkg().mla_tree_mask(s["parents"], s["qo"], s["host"]["words"], kv_lens=s["kv"])


def _own_commit(s):
    _pkg().mla_tree_commit(s["cache"], s["table"], s["seq"], s["paths"], s["acc"])
    return s["cache"]


def _plain_attention(s):
    c, h = s["case"], s["host"]
    heads, bs = c["heads"], c["block"]
    q, flat = s["q"], s["cache"].view(-1, E)
    o = torch.empty((q.shape[0], heads, DV), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((q.shape[0], heads), dtype=torch.float32, device="cuda")
    for r in range(c["batch"]):
        t0, t1, kv = int(h["qo"][r]), int(h["qo"][r + 1]), int(h["kv"][r])
        n = t1 - t0
        pos = torch.arange(kv, device="cuda")
        keys = flat[s["table"][r].long()[pos // bs] * bs + pos % bs].float()
        x = (q[t0:t1].float().reshape(n * heads, E) @ keys.T) * SM_SCALE
        if c["cap"] > 0:
            x = c["cap"] * torch.tanh(x / c["cap"])
        node = pos - (kv - n)                                   # negative: the context
        if c["tree"]:
            word = s["mask"][t0:t1][:, node.clamp(min=0) >> 6]
            seen = ((word >> (node.clamp(min=0) & 63)) & 1).bool() | (node < 0)
        else:
            seen = node[None, :] <= torch.arange(n, device="cuda")[:, None]
        x = x.view(n, heads, kv).masked_fill(~seen[:, None, :], float("-inf"))
        top = x.amax(dim=-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        p = torch.exp(x - top)
        tot = p.sum(dim=-1, keepdim=True)
        acc = (p.view(n * heads, kv) @ keys[:, :DV]).view(n, heads, DV)
        o[t0:t1] = torch.where(tot > 0, acc / tot, torch.zeros_like(acc)).to(torch.bfloat16)
        lse[t0:t1] = (top + torch.log(tot))[..., 0]
    return o, lse


def _plain_update(seq, new, table, held, free, count, bs, tokens):
    seq, new, held0 = seq.long(), new.long(), held.long()
    target = (seq + new + bs - 1) // bs
    rel, need = (held0 - target).clamp(min=0), (target - held0).clamp(min=0)
    rel_end, need_end = rel.cumsum(0), need.cumsum(0)
    base = count.long()
    top = base + rel_end[-1]
    granted = need_end <= top
    after = torch.where(need > 0, torch.where(granted, target, held0), target)
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    # surplus blocks go on the free stack, so that the next to be taken is the first given back
    out = (j >= target[:, None]) & (j < held0[:, None])
    k = (rel_end - rel)[:, None] + j - target[:, None]
    free[(top - 1 - k)[out]] = table[out]
    table[out] = -1
    take = (j >= held0[:, None]) & (j < after[:, None])
    k = (need_end - need)[:, None] + j - held0[:, None]
    table[take] = free[(top - 1 - k)[take]]
    held.copy_(after)
    count.copy_(top - torch.where(granted, need, torch.zeros_like(need)).sum())
    qo = torch.zeros(len(seq) + 1, dtype=torch.int32, device="cuda")
    qo[1:] = new.cumsum(0)
    t = torch.arange(tokens, device="cuda")
    r = torch.searchsorted(qo[1:].long(), t, right=True)
    live = r < len(seq)
    r = r.clamp(max=len(seq) - 1)
    pos = seq[r] + t - qo[r]
    live &= pos // bs < table.shape[1]
    blk = table[r, (pos // bs).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & (blk >= 0), blk * bs + pos % bs, torch.full_like(pos, -1))
    return qo, (seq + new).int(), slots


def _plain_tables(s):
    bs, tokens = s["case"]["block"], s["host"]["tokens"]
    state = [s["table"], s["held"], s["free"], s["count"]]
    out = _plain_update(s["seq"], s["new"], *state, bs, tokens)
    _plain_update(s["seq"], s["zero"], *state, bs, 0)
    return list(out) + state


def _plain_mask(s):
    qo, kv = s["qo"].long(), s["kv"].long()
    n = qo[1:] - qo[:-1]
    width, words = s["host"]["words"] * 64, s["host"]["words"]
    batch, total = len(n), s["parents"].shape[0]
    r = torch.searchsorted(qo[1:], torch.arange(total, device="cuda"), right=True)
    i = torch.arange(total, device="cuda") - qo[r]
    parents = torch.full((batch, width), -1, dtype=torch.int64, device="cuda")
    parents[r, i] = s["parents"].long()
    seen = torch.eye(width, dtype=torch.bool, device="cuda").repeat(batch, 1, 1)
    depth = torch.zeros((batch, width), dtype=torch.int64, device="cuda")
    rows = torch.arange(batch, device="cuda")
    for c in range(1, int(np.diff(s["host"]["qo"]).max())):
        p = parents[:, c]
        has, up = p >= 0, p.clamp(min=0)
        seen[:, c] |= seen[rows, up] & has[:, None]
        depth[:, c] = torch.where(has, depth[rows, up] + 1, torch.zeros_like(p))
    bit = torch.arange(64, device="cuda")
    packed = (seen.view(batch, width, words, 64).long() << bit).sum(-1)
    return packed[r, i].contiguous(), ((kv - n)[r] + depth[r, i]).int()


def _plain_commit(s):
    bs, cache, paths = s["case"]["block"], s["cache"], s["paths"].long()
    i = torch.arange(paths.shape[1], device="cuda")[None, :]
    live = i < s["acc"][:, None]
    base = s["seq"].long()[:, None]

    def slot(pos):
        return torch.gather(s["table"].long(), 1, (pos // bs).clamp(max=s["table"].shape[1] - 1)) * bs + pos % bs

    src, dst = slot(base + paths.clamp(min=0))[live], slot(base + i.expand_as(paths).clamp(max=s["case"]["nodes"] - 1))[live]
    flat = cache.view(cache.shape[0], -1, E)
    flat[:, dst] = flat[:, src]
    return cache


_run_plain = {"attention": _plain_attention, "tables": _plain_tables, "mask": _plain_mask, "commit": _plain_commit}
_run_own = {"attention": _own_attention, "tables": _own_tables, "mask": _own_mask, "commit": _own_commit}


# ------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    h = _host(case, seed)
    return {"attention": _exact_attention, "tables": _exact_tables, "mask": _exact_mask,
            "commit": _exact_commit}[case["op"]](case, h, seed)


def _exact_attention(case, h, seed):
    big = _big(case, h, seed)
    heads, bs = case["heads"], case["block"]
    rows = big["cache"].view(-1, E)
    out_o, out_l = [], []
    for r in range(case["batch"]):
        t0, t1, kv = int(h["qo"][r]), int(h["qo"][r + 1]), int(h["kv"][r])
        n = t1 - t0
        slots = (h["table"][r].astype(np.int64)[:, None] * bs + np.arange(bs)[None, :]).reshape(-1)[:kv]
        c = rows[torch.from_numpy(slots).to("cuda")].double()
        for i in range(n):
            kin = [j for j in range(n)
                   if ((int(h["mask"][t0 + i, j >> 6]) >> (j & 63)) & 1 if case["tree"] else j <= i)]
            mine = c if len(kin) == n else torch.cat([c[:kv - n], c[torch.tensor(kin, device="cuda") + kv - n]])
            z = torch.einsum("he,ke->hk", big["q"][t0 + i].double(), mine) * SM_SCALE
            if case["cap"] > 0:
                z = case["cap"] * torch.tanh(z / case["cap"])
            norm = torch.logsumexp(z, dim=1)
            out_o.append(torch.einsum("hk,kd->hd", torch.exp(z - norm[:, None]), mine[:, :DV]))
            out_l.append(norm)
    return torch.stack(out_o), torch.stack(out_l)


def _exact_tables(case, h, seed):
    bs = case["block"]
    table, stack = h["table"].copy(), [int(x) for x in h["free"][:int(h["count"][0])]]
    slots, qo = [], [0]
    for r in range(case["batch"]):
        seq, new = int(h["seq"][r]), int(h["new"][r])
        for j in range(int(h["held"][r]), -(-(seq + new) // bs)):
            table[r, j] = stack.pop()
        p = np.arange(seq, seq + new)
        slots.append(table[r, p // bs].astype(np.int64) * bs + p % bs)
        qo.append(qo[-1] + new)
    slots.append(np.full(h["tokens"] - qo[-1], -1, dtype=np.int64))
    back = [np.array(qo, np.int32), h["seq"] + h["new"], np.concatenate(slots), h["table"], h["held"], h["free"],
            h["count"]]   # rolled back: as it was
    return [torch.from_numpy(np.ascontiguousarray(x)).to("cuda") for x in back]


def _exact_mask(case, h, seed):
    bits, depth = _ancestors(h["parents"], h["qo"])
    nodes = np.diff(h["qo"])
    pos = np.repeat(h["kv"] - nodes, nodes) + depth
    return torch.from_numpy(bits.copy()).to("cuda"), torch.from_numpy(pos.astype(np.int32)).to("cuda")


def _exact_commit(case, h, seed):
    cache = _big(case, h, seed)["cache"]
    out = cache.clone()
    bs = case["block"]
    for r in range(case["batch"]):
        for i in range(int(h["acc"][r])):
            a, b = int(h["seq"][r]) + int(h["paths"][r, i]), int(h["seq"][r]) + i
            out[:, h["table"][r, b // bs], b % bs] = cache[:, h["table"][r, a // bs], a % bs]
    return out


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(one, work(one))
