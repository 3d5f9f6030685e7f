"""What is timed of the 4-bit latent cache and of the ends of a speculative-decoding step.

Four operators: ``mla_cache_append`` (new tokens' latents normalised, their rotary part rotated,
both stored in a paged cache of bf16, fp8 or 4-bit entries, and the queries rotated on the way),
``mla_gather_latent_fp4`` (prefix rows out of a 4-bit cache), ``mla_tree_attention_fp4`` (drafted
or single new tokens over a 4-bit cache, absorbed-weight form) and ``mla_tree_verify`` (drafted
trees against the target's probabilities, from given random numbers).  A case is a dict of plain
values; ``run`` makes one pass over a prepared state, in elementary torch operations or, where
``own`` is true, with the package's kernels; ``exact`` computes the same outputs apart from both,
in 64 bits.

A 4-bit entry has 400 bytes: [0, 256) 512 latent codes in e2m1 (1 sign, 2 exponent, 1 mantissa
bit), eight to a 32-bit little-endian word, of which values 0, 2, 4, 6 are the low half's nibbles
from bit 0 up and 1, 3, 5, 7 the high half's; [256, 384) the rotary part, 64 bf16; [384, 400)
a scale byte b, 2^(b - 127), for each 32 latents.  An fp8 entry has 648: 512 e4m3 codes, 64 bf16,
8 scale bytes for 64 latents each.
"""
import random
import zlib

import numpy as np
import torch

own = False

E, DV, ROPE = 576, 512, 64  # cache row: 512 latent + 64 rotary values; attention's values are the first 512
SM_SCALE = 192 ** -0.5      # the head dim before absorption is 128 + 64
EPS = 1e-6

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
        # One request's next token over a short context, 16 heads (the heads of one GPU of eight): the
        # latency of a call.
        {"name": "attn4_1x1_over_700_h16", "op": "attention", "nodes_lo": 1, "nodes": 1, "batch": 1, "ctx_lo": 700, "ctx": 700,
         "heads": 16, "block": 64, "tree": False, "cap": 0.0},
        # Single tokens of many requests, 16 heads: what a small cache is for, bound by reading it.
        {"name": "attn4_64x1_over_8192_h16", "op": "attention", "nodes_lo": 1, "nodes": 1, "batch": 64, "ctx_lo": 8192,
         "ctx": 8192, "heads": 16, "block": 64, "tree": False, "cap": 0.0},
        # Single tokens with every head on one GPU, ragged contexts.
        {"name": "attn4_32x1_ragged_h128", "op": "attention", "nodes_lo": 1, "nodes": 1, "batch": 32, "ctx_lo": 129, "ctx": 16001,
         "heads": 128, "block": 64, "tree": False, "cap": 0.0},
        # Ragged trees over small pages, odd counts, capped logits.
        {"name": "attn4_9x37_ragged_h16_page16", "op": "attention", "nodes_lo": 3, "nodes": 37, "batch": 9, "ctx_lo": 1,
         "ctx": 5001, "heads": 16, "block": 16, "tree": True, "cap": 30.0},
        # The batch that prefill runs at 128 heads, verifying 16 drafts per request: compute bound.
        {"name": "attn4_32x16_over_8192_h128", "op": "attention", "nodes_lo": 16, "nodes": 16, "batch": 32, "ctx_lo": 8192,
         "ctx": 8192, "heads": 128, "block": 64, "tree": True, "cap": 0.0},
        # A decoding step's new rows into a 4-bit cache, its queries rotated, and the rows read back.
        {"name": "append_64x1_fp4_h16", "op": "append", "format": "fp4", "batch": 64, "seq_lo": 50, "seq": 9000, "new_lo": 1,
         "new": 1, "heads": 16, "norm": True, "interleaved": True, "block": 64},
        # Ragged prompts into an fp8 cache, keys only, and the rows read back.
        {"name": "append_5x2049_fp8", "op": "append", "format": "fp8", "batch": 5, "seq_lo": 0, "seq": 4001, "new_lo": 130,
         "new": 2049, "heads": 0, "norm": True, "interleaved": False, "block": 24},
        # The new tokens of the chunked-prefix batch at 128 heads into the bf16 cache.
        {"name": "append_4x2048_bf16_h128", "op": "append", "format": "bf16", "batch": 4, "seq_lo": 8192, "seq": 8192,
         "new_lo": 2048, "new": 2048, "heads": 128, "norm": True, "interleaved": True, "block": 64},
        # A short prefix out of a 4-bit cache, and the chunked-prefix batch's whole one.
        {"name": "gather4_3x500_page16", "op": "gather", "batch": 3, "rows_lo": 1, "rows": 500, "start": 37, "block": 16},
        {"name": "gather4_4x8192", "op": "gather", "batch": 4, "rows_lo": 8192, "rows": 8192, "start": 0, "block": 64},
        # One request's chain of drafts, given tokens, a small vocabulary: the latency of a call.
        {"name": "verify_1x5_given", "op": "verify", "batch": 1, "nodes_lo": 5, "nodes": 5, "vocab": 32003, "tree": False,
         "drawn": False, "type": "fp32"},
        # A batch of trees whose drafts were drawn from the draft model's probabilities.
        {"name": "verify_64x16_drawn", "op": "verify", "batch": 64, "nodes_lo": 5, "nodes": 16, "vocab": 131072, "tree": True,
         "drawn": True, "type": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "gather", "verify", "verify"])
    block = rng.choice([16, 32, 64, 64, 128, 24, 1, 7])
    if op == "attention":
        heads = rng.choice([1, 5, 8, 16, 16, 32, 48, 64, 128, 128])
        batch = _log(rng, 1, 96)
        tree = rng.random() < 0.5
        n1 = _log(rng, 1, 80) if tree or rng.random() < 0.2 else 1
        n0 = rng.randint(1, n1)
        c1 = _log(rng, 1, 60000)
        c0 = rng.randint(max(1, c1 // 20), c1)
        # no dearer than the largest listed case, in operations and in cached tokens
        while batch > 1 and (batch * n1 * heads * (c1 + n1) > 32 * 16 * 128 * 8192 or batch * c1 > 500000):
            batch = max(1, batch // 2)
        while n1 > 1 and n1 * heads * (c1 + n1) * batch > 32 * 16 * 128 * 8192:
            n1, n0 = max(1, n1 // 2), 1
        return {"op": op, "nodes_lo": n0, "nodes": n1, "batch": batch, "ctx_lo": c0, "ctx": c1, "heads": heads, "block": block,
                "tree": tree, "cap": rng.choice([0.0, 0.0, 30.0])}
    if op == "append":
        n1 = _log(rng, 1, 4000)
        batch = max(1, min(_log(rng, 1, 300), 8192 // n1))
        s1 = rng.choice([0, _log(rng, 1, 30000)])
        return {"op": op, "format": rng.choice(["bf16", "fp8", "fp4", "fp4"]), "batch": batch, "seq_lo": rng.randint(0, s1),
                "seq": s1, "new_lo": rng.randint(1, n1), "new": n1, "heads": rng.choice([0, 1, 5, 16, 64, 128]),
                "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.5, "block": block}
    if op == "gather":
        r1 = _log(rng, 1, 30000)
        return {"op": op, "batch": max(1, min(_log(rng, 1, 200), 32768 // r1)), "rows_lo": rng.randint(0, r1), "rows": r1,
                "start": rng.choice([0, 1, 100, 3001]), "block": block}
    n1 = _log(rng, 1, 40)
    vocab = _log(rng, 1000, 131072)
    return {"op": op, "batch": max(1, min(_log(rng, 1, 64), 1024 // n1)), "nodes_lo": rng.randint(1, n1), "nodes": n1, "vocab": vocab,
            "tree": rng.random() < 0.6, "drawn": rng.random() < 0.6, "type": rng.choice(["fp32", "fp32", "bf16"])}


def _mean(case, what):
    return (case[what + "_lo"] + case[what]) / 2


def _words(nodes):
    return (nodes + 63) // 64


_ENTRY = {"bf16": 1152, "fp8": 648, "fp4": 400}


def work(case):
    b = case["batch"]
    if case["op"] == "attention":
        n, ctx = _mean(case, "nodes"), _mean(case, "ctx")
        t = b * n * case["heads"]
        mask = b * n * 8 * _words(case["nodes"]) if case["tree"] else 0
        return {"bytes": int(b * (ctx + n) * (400 + 4 / case["block"]) + t * (E * 2 + DV * 2 + 4) + mask + 8 * b),
                "flops": int(2 * t * (ctx + 1) * (E + DV))}
    if case["op"] == "append":
        t = b * _mean(case, "new")
        entry = _ENTRY[case["format"]]
        back = 0 if case["format"] == "bf16" else entry + E * 2   # what is read back as values
        return {"bytes": int(t * (E * 2 + entry + back + 4 + 8 + 4 * ROPE + case["heads"] * ROPE * 2 * 2)), "flops": int(t * DV * 4)}
    if case["op"] == "gather":
        return {"bytes": int(b * _mean(case, "rows") * (400 + E * 2 + 4 / case["block"])), "flops": 0}
    # the last node's row of a request, and a few numbers of each node
    size = 4 if case["type"] == "fp32" else 2
    return {"bytes": int(b * case["vocab"] * size * (2 if case["drawn"] else 1) + b * _mean(case, "nodes") * 20), "flops": 0}


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
    """Parents of every request's nodes (-1 for node 0), each before its child; deep and bushy
    trees both occur, as drafting a few best continuations makes them."""
    out = []
    for n in nodes:
        reach = int(rng.integers(1, 9))
        p = np.array([int(rng.integers(max(0, i - reach), max(1, i))) for i in range(int(n))], dtype=np.int32)
        p[:1] = -1
        out.append(p)
    return np.concatenate(out) if out else np.zeros(0, np.int32)


def _ancestors(parents, qo):
    """Host visibility of every node: its own bit and its ancestors', int64 [T, words]."""
    words = _words(int(np.diff(qo).max(initial=1)))
    bits = np.zeros((len(parents), words), dtype=np.uint64)
    for r in range(len(qo) - 1):
        for t in range(int(qo[r]), int(qo[r + 1])):
            i, p = t - int(qo[r]), int(parents[t])
            if p >= 0:
                bits[t] = bits[qo[r] + p]
            bits[t, i >> 6] |= np.uint64(1) << np.uint64(i & 63)
    return bits.view(np.int64)


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
    return table, total


def _host(case, seed):
    """Lengths, tables, trees: everything but the large tensors, on the host."""
    rng = np.random.default_rng([seed, 78])
    # lengths belong to the case, so that every seed's outputs have the same shapes
    sizes = np.random.default_rng(zlib.crc32(repr(sorted((k, v) for k, v in case.items() if k != "name")).encode()))
    h = {"op": case["op"]}
    if case["op"] == "attention":
        nodes, ctx = _lengths(sizes, case, "nodes"), _lengths(sizes, case, "ctx")
        h["qo"], h["kv"] = _indptr(nodes), (nodes + ctx).astype(np.int32)
        h["table"], h["blocks"] = _paged(rng, nodes + ctx, case["block"])
        if case["tree"]:
            h["mask"] = _ancestors(_trees(rng, nodes), h["qo"])
    elif case["op"] == "append":
        seq, new, bs = _lengths(sizes, case, "seq"), _lengths(sizes, case, "new"), case["block"]
        h["table"], h["blocks"] = _paged(rng, seq + new, bs)
        h["cu"], h["starts"] = _indptr(new), seq.astype(np.int32)
        r = np.repeat(np.arange(len(new)), new)
        pos = seq[r] + np.arange(int(new.sum())) - h["cu"][r]
        slots = h["table"][r, pos // bs].astype(np.int64) * bs + pos % bs
        h["live"] = len(pos)
        # the padded rows of a captured step: no slot, and positions that mean nothing
        h["slots"] = np.concatenate([slots, np.full(3, -1)]).astype(np.int64)
        h["positions"] = np.concatenate([pos, [0, -7, 1 << 30]]).astype(np.int32)
        h["reach"] = int((seq + new).max())
    elif case["op"] == "gather":
        rows, bs = _lengths(sizes, case, "rows"), case["block"]
        h["table"], h["blocks"] = _paged(rng, rows + case["start"], bs)
        h["cu"], h["starts"] = _indptr(rows), np.full(len(rows), case["start"], dtype=np.int32)
    else:
        nodes = _lengths(sizes, case, "nodes")
        h["qo"] = _indptr(nodes)
        if case["tree"]:
            h["parents"] = _trees(rng, nodes)
        else:
            h["parents"] = np.concatenate([np.arange(n) - 1 for n in nodes]).astype(np.int32)
        total = int(h["qo"][-1])
        h["u"] = rng.random(total, dtype=np.float32)
        h["u_last"] = rng.random(case["batch"], dtype=np.float32)
    return h


def _big(case, h, seed):
    """The large tensors, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed * 2 + 1)
    bf = dict(dtype=torch.bfloat16, device="cuda", generator=g)
    if case["op"] == "attention":
        rows = h["blocks"] * case["block"]
        # latents behind a norm are about N(0, 1); here they are rounded as the cache holds them
        entries = _encode4(torch.randn((rows, DV), device="cuda", generator=g), torch.randn((rows, ROPE), **bf))
        return {"cache": entries.view(h["blocks"], case["block"], 400),
                "q": torch.randn((int(h["qo"][-1]), case["heads"], E), **bf)}
    if case["op"] == "append":
        t = len(h["slots"])
        out = {"latent": torch.randn((t, E + 64), **bf) * 1.7, "weight": 1 + torch.randn(DV, **bf) / 8}
        if case["heads"]:
            out["q"] = torch.randn((t, case["heads"], 192), **bf)
        return out
    if case["op"] == "gather":
        rows = h["blocks"] * case["block"]
        entries = _encode4(torch.randn((rows, DV), device="cuda", generator=g), torch.randn((rows, ROPE), **bf))
        return {"cache": entries.view(h["blocks"], case["block"], 400)}
    t, v = len(h["u"]), case["vocab"]
    logits = torch.randn((t, v), device="cuda", generator=g) * 2.5
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits + 0.7 * torch.randn((t, v), device="cuda", generator=g), -1)
    # what a drafting model proposes after each node's parent: drawn, or its best continuations in turn
    qo, parents = torch.from_numpy(h["qo"]).cuda().long(), torch.from_numpy(h["parents"]).cuda().long()
    first = torch.repeat_interleave(qo[:-1], qo[1:] - qo[:-1])
    up = first + parents.clamp(min=0)
    if case["drawn"]:
        tokens = torch.multinomial(draft[up], 1, generator=g)[:, 0]
    else:
        rank = torch.from_numpy(_sibling_ranks(h)).cuda()
        tokens = torch.topk(draft[up], int(rank.max()) + 1, dim=-1).indices.gather(1, rank[:, None])[:, 0]
    kind = torch.float32 if case["type"] == "fp32" else torch.bfloat16
    out = {"tokens": tokens.int(), "target": target.to(kind)}
    if case["drawn"]:
        out["draft"] = draft.to(kind)
    return out


def _sibling_ranks(h):
    """How many earlier nodes of its request have a node's parent."""
    seen, out = {}, []
    for r in range(len(h["qo"]) - 1):
        for t in range(int(h["qo"][r]), int(h["qo"][r + 1])):
            k = (r, int(h["parents"][t]))
            out.append(seen.get(k, 0))
            seen[k] = out[-1] + 1
    return np.array(out, dtype=np.int64)


def _cos_sin(positions):
    """cos and sin of position * 10000^(-i / 32), i < 32: [positions, 64] fp32."""
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([torch.cos(angle), torch.sin(angle)], dim=-1).float()


def prepare(case, seed):
    h = _host(case, seed)
    s = {"case": case, "host": h}
    for k, v in h.items():
        if isinstance(v, np.ndarray):
            s[k] = torch.from_numpy(v.copy()).to("cuda")
    s.update(_big(case, h, seed))
    if case["op"] == "append":
        s["cos_sin"] = _cos_sin(h["reach"])
        kind = torch.bfloat16 if case["format"] == "bf16" else torch.uint8
        width = E if case["format"] == "bf16" else _ENTRY[case["format"]]
        s["cache"] = torch.zeros((h["blocks"], case["block"], width), dtype=kind, device="cuda")
        s["latent"] = s["latent"][:, 64:]      # part of a wider projection's rows
        if case["heads"]:
            s["q_out"] = torch.zeros_like(s["q"])[..., 128:]
            s["q"] = s["q"][..., 128:]
    return s


# ------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_attention(s):
    c = s["case"]
    return _pkg().mla_tree_attention_fp4(s["q"], s["cache"], s["table"], s["qo"], s["kv"], s.get("mask"),
                                         sm_scale=SM_SCALE, logits_soft_cap=c["cap"])


def _own_append(s):
    m, c, h = _pkg(), s["case"], s["host"]
    m.mla_cache_append(s["cache"], s["latent"], s["slots"], s["positions"], s["cos_sin"],
                       norm_weight=s["weight"] if c["norm"] else None, norm_eps=EPS, interleaved=c["interleaved"],
                       q_rope=s.get("q"), q_out=s.get("q_out"))
    out = {}
    if c["heads"]:
        out["q"] = s["q_out"]
    if c["format"] == "bf16":
        out["cache"] = s["cache"]
    else:
        gather = m.mla_gather_latent_fp4 if c["format"] == "fp4" else m.mla_gather_latent_fp8
        out["rows"] = gather(s["cache"], s["table"], s["cu"], s["starts"], h["live"])
    return out


def _own_gather(s):
    return _pkg().mla_gather_latent_fp4(s["cache"], s["table"], s["cu"], s["starts"], int(s["host"]["cu"][-1]))


def _own_verify(s):
    return _pkg().mla_tree_verify(s["target"], s["tokens"], s["qo"], s["u"], s["u_last"], s["case"]["nodes"],
                                  parents=s["parents"] if s["case"]["tree"] else None, draft_probs=s.get("draft"))


def _scale_exponent(amax, top):
    """The least k with amax <= 1.75 * 2^(top + k), -127 <= k: 2^k is a group's scale."""
    m, e = torch.frexp(amax)
    k = e - 1 + (m > 0.875) - top
    return torch.where(amax > 0, k, torch.full_like(k, -127)).clamp(min=-127)


def _encode4(x, rope):
    """Entries [T, 400] of latents [T, 512] fp32 and rotary parts [T, 64] bf16."""
    t = x.shape[0]
    x = x.reshape(t, 16, 32)
    k = _scale_exponent(x.abs().amax(-1), 2)
    y = torch.ldexp(x, -k[..., None])
    a = y.abs()
    # to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6, ties to the even code
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)).byte() | ((y < 0).byte() << 3)
    code = code.view(t, 64, 2, 2, 2).permute(0, 1, 4, 2, 3)       # word, half, byte, nibble
    packed = (code[..., 0] | (code[..., 1] << 4)).reshape(t, 256)
    return torch.cat([packed, rope.contiguous().view(torch.uint8), (k + 127).byte()], dim=-1)


def _decode4(entries):
    """Values [..., 576] fp32 of entries [..., 400]."""
    lead = entries.shape[:-1]
    e = entries.reshape(-1, 400)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=e.device)
    codes = torch.stack([e[:, :256] & 15, e[:, :256] >> 4], dim=-1).view(-1, 64, 2, 2, 2).permute(0, 1, 3, 4, 2)
    lat = grid[codes.reshape(-1, 16, 32).int()] * torch.exp2(e[:, 384:].float() - 127)[..., None]
    rope = e[:, 256:384].contiguous().view(torch.bfloat16).float()
    return torch.cat([lat.reshape(-1, DV), rope], dim=-1).view(*lead, E)


def _rows_of(table, r, pos, bs):
    """Flat cache rows of positions `pos` of requests `r`."""
    return table[r, (pos // bs).clamp(max=table.shape[1] - 1)].long().clamp(min=0) * bs + pos % bs


def _plain_attention(s):
    c, h = s["case"], s["host"]
    heads, bs, batch = c["heads"], c["block"], c["batch"]
    kv, qo = s["kv"].long(), s["qo"].long()
    n = qo[1:] - qo[:-1]
    most, longest = int(np.diff(h["qo"]).max()), int(h["kv"].max())
    pos = torch.arange(longest, device="cuda")
    r = torch.arange(batch, device="cuda")
    # every request padded to the longest
    keys = _decode4(s["cache"].view(-1, 400)[_rows_of(s["table"], r[:, None], pos[None, :], bs)])
    i = torch.arange(most, device="cuda")
    rows = (qo[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(batch, most * heads, E)
    x = torch.bmm(q, keys.transpose(1, 2)) * SM_SCALE
    if c["cap"] > 0:
        x = c["cap"] * torch.tanh(x / c["cap"])
    node = pos[None, :] - (kv - n)[:, None]                      # negative: the context
    if c["tree"]:
        j = node.clamp(min=0, max=64 * s["mask"].shape[1] - 1)
        word = torch.gather(s["mask"][rows], 2, (j >> 6)[:, None, :].expand(-1, most, -1))
        seen = ((word >> (j & 63)[:, None, :]) & 1).bool() | (node < 0)[:, None, :]
    else:
        seen = node[:, None, :] <= i[None, :, None]
    seen = seen & (pos[None, :] < kv[:, None])[:, None, :]
    x = x.view(batch, most, heads, longest).masked_fill_(~seen[:, :, None, :], float("-inf"))
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    tot = p.sum(dim=-1, keepdim=True)
    acc = torch.bmm(p.view(batch, most * heads, longest), keys[..., :DV]).view(batch, most, heads, DV)
    o = torch.where(tot > 0, acc / tot, torch.zeros_like(acc)).to(torch.bfloat16)
    lse = (top + torch.log(tot))[..., 0]
    live = i[None, :] < n[:, None]
    return o[live], lse[live]


def _rotate(x, cs, interleaved):
    """x [..., 64] fp32 rotated by the angles of cs [..., 64] (32 cosines, 32 sines)."""
    cos, sin = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    y = [a * cos - b * sin, b * cos + a * sin]
    return torch.stack(y, dim=-1).flatten(-2) if interleaved else torch.cat(y, dim=-1)


def _plain_append(s):
    c, live = s["case"], s["host"]["live"]
    slots = s["slots"][:live]                                    # (the others are padding)
    x = s["latent"][:live].float()
    cs = s["cos_sin"][s["positions"][:live].long()]
    lat = x[:, :DV]
    if c["norm"]:
        lat = lat * torch.rsqrt((lat * lat).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    rope = _rotate(x[:, DV:], cs, c["interleaved"]).to(torch.bfloat16)
    out = {}
    if c["heads"]:
        s["q_out"][:live] = _rotate(s["q"][:live].float(), cs[:, None, :], c["interleaved"]).to(torch.bfloat16)
        out["q"] = s["q_out"]
    if c["format"] == "bf16":
        s["cache"].view(-1, E)[slots] = torch.cat([lat.to(torch.bfloat16), rope], dim=-1)
        out["cache"] = s["cache"]
    elif c["format"] == "fp4":
        flat = s["cache"].view(-1, 400)
        flat[slots] = _encode4(lat, rope)
        out["rows"] = _decode4(flat[slots]).to(torch.bfloat16)
    else:
        g = lat.reshape(live, 8, 64)
        k = _scale_exponent(g.abs().amax(-1), 8)
        code = torch.ldexp(g, -k[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(live, DV)
        flat = s["cache"].view(-1, 648)
        flat[slots] = torch.cat([code, rope.view(torch.uint8), (k + 127).byte()], dim=-1)
        back = flat[slots]
        val = back[:, :DV].contiguous().view(torch.float8_e4m3fn).float().view(live, 8, 64)
        val = val * torch.exp2(back[:, 640:].float() - 127)[..., None]
        out["rows"] = torch.cat([val.view(live, DV).to(torch.bfloat16), back[:, DV:640].contiguous().view(torch.bfloat16)], dim=-1)
    return out


def _plain_gather(s):
    cu, total = s["cu"].long(), int(s["host"]["cu"][-1])
    t = torch.arange(total, device="cuda")
    r = torch.searchsorted(cu[1:], t, right=True)
    pos = s["starts"][r].long() + t - cu[r]
    return _decode4(s["cache"].view(-1, 400)[_rows_of(s["table"], r, pos, s["case"]["block"])]).to(torch.bfloat16)


def _plain_verify(s):
    c, qo = s["case"], s["qo"].long()
    batch, most, total = c["batch"], c["nodes"], s["tokens"].shape[0]
    n = qo[1:] - qo[:-1]
    r = torch.repeat_interleave(torch.arange(batch, device="cuda"), n, output_size=total)
    first = qo[r]
    up = first + s["parents"].long().clamp(min=0)                # the parent's row
    root = s["parents"] < 0
    tok, u = s["tokens"].long(), s["u"].double()
    p_t = s["target"][up, tok].double()
    # earlier nodes of the same parent
    j = torch.arange(most, device="cuda")
    other = (first[:, None] + j).clamp(max=total - 1)
    before = (other < torch.arange(total, device="cuda")[:, None]) & (j < n[r][:, None]) & (up[other] == up[:, None]) & ~root[other] & ~root[:, None]
    rank = before.sum(-1)
    if c["drawn"]:
        q_t = s["draft"][up, tok].double()
        ok = (u * q_t < p_t) & (rank == 0)
        times = torch.zeros(total, dtype=torch.float64, device="cuda")       # of the draft taken off at each node
        times[up[(rank == 0) & ~root]] = 1
        for k in range(1, int(rank.max()) + 1):                  # a sibling at a time: each needs the sum that the last left
            mine = torch.nonzero(rank == k)[:, 0]
            at = up[mine]
            room = (s["target"][at].double() - times[at, None] * s["draft"][at].double()).clamp(min=0).sum(-1)
            ok[mine] = u[mine] * q_t[mine] * room < (p_t[mine] - times[at] * q_t[mine]).clamp(min=0)
            times[at] += room
    else:
        same = before & (tok[other] == tok[:, None])
        fresh = ~same.any(-1)
        gone = (before & fresh[other]).double() * p_t[other]
        ok = (u * (1 - gone.sum(-1)) < p_t) & fresh
    ok = ok & ~(before & ok[other]).any(-1)                      # the first that passes
    ok = torch.where(root, torch.arange(total, device="cuda") == first, ok)
    jump = torch.where(root, torch.arange(total, device="cuda"), up)
    for _ in range(max(1, (most - 1).bit_length())):             # and every ancestor too
        ok = ok & ok[jump]
        jump = jump[jump]
    order = torch.where(ok, torch.arange(total, device="cuda") - first, torch.full_like(first, most))
    grid = torch.full((batch, most), most, dtype=torch.int64, device="cuda")
    grid[r, torch.arange(total, device="cuda") - first] = order
    path = grid.sort(-1).values
    counts = (path < most).sum(-1)
    last = qo[:-1] + path.gather(1, (counts - 1)[:, None])[:, 0]
    rest = s["target"][last].double()
    if c["drawn"]:
        left = (rest - times[last, None] * s["draft"][last].double()).clamp(min=0)
    else:
        left = rest.clone()
        child = ~root & (up == last[r])
        left[r[child], tok[child]] = 0
    rest = torch.where(left.sum(-1, keepdim=True) > 0, left, rest).cumsum(-1)
    token = torch.searchsorted(rest, (s["u_last"].double() * rest[:, -1])[:, None], right=True)[:, 0]
    path = torch.where(path < most, path, torch.full_like(path, -1))
    return path.int(), counts.int(), token.int()


_run_plain = {"attention": _plain_attention, "append": _plain_append, "gather": _plain_gather, "verify": _plain_verify}
_run_own = {"attention": _own_attention, "append": _own_append, "gather": _own_gather, "verify": _own_verify}


# ------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    h = _host(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "gather": _exact_gather,
            "verify": _exact_verify}[case["op"]](case, h, seed)


def _values64(entries):
    """fp64 values of entries [T, 400], bit by bit."""
    words = entries[:, :256].contiguous().view(torch.int32).long()
    out = torch.empty((entries.shape[0], E), dtype=torch.float64, device="cuda")
    for v in range(8):
        code = words >> (16 * (v % 2) + 4 * (v // 2))
        e, m = (code >> 1) & 3, (code & 1).double()
        mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2((e - 1).double()))
        scale = torch.exp2(entries[:, 384:].double() - 127).repeat_interleave(4, dim=1)
        out[:, v:DV:8] = mag * (1 - 2 * ((code >> 3) & 1)) * scale
    out[:, DV:] = entries[:, 256:384].contiguous().view(torch.bfloat16).double()
    return out


def _exact_attention(case, h, seed):
    big = _big(case, h, seed)
    bs = case["block"]
    flat = big["cache"].view(-1, 400)
    out_o, out_l = [], []
    for r in range(case["batch"]):
        t0, t1, kv = int(h["qo"][r]), int(h["qo"][r + 1]), int(h["kv"][r])
        n = t1 - t0
        slots = (h["table"][r].astype(np.int64)[:, None] * bs + np.arange(bs)[None, :]).reshape(-1)[:kv]
        c = _values64(flat[torch.from_numpy(slots).to("cuda")])
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


def _turn64(x, pos, table, interleaved):
    out = x.double().clone()
    cs = table.double()[pos]
    for i in range(32):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        c, s = cs[:, i], cs[:, 32 + i]
        while c.dim() < x.dim() - 1:
            c, s = c[:, None], s[:, None]
        u, v = x[..., a].double(), x[..., b].double()
        out[..., a], out[..., b] = u * c - v * s, u * s + v * c
    return out


def _grid64(bits_e, bits_m, bias, top):
    """Every magnitude of a small float type, in order of its codes."""
    vals = [m / (1 << bits_m) * 2.0 ** (1 - bias) if e == 0 else (1 + m / (1 << bits_m)) * 2.0 ** (e - bias)
            for e in range(1 << bits_e) for m in range(1 << bits_m)]
    return torch.tensor(vals[:top], dtype=torch.float64, device="cuda")


def _exact_append(case, h, seed):
    big, live = _big(case, h, seed), h["live"]
    x = big["latent"][:live, 64:].double()
    lat = x[:, :DV]
    if case["norm"]:
        lat = lat / torch.sqrt((lat * lat).sum(-1, keepdim=True) / DV + EPS) * big["weight"].double()
    pos = torch.from_numpy(h["positions"][:live].astype(np.int64)).to("cuda")
    table = _cos_sin(h["reach"])
    rope = _turn64(x[:, DV:], pos, table, case["interleaved"])
    out = {}
    if case["heads"]:
        q = torch.zeros((len(h["slots"]), case["heads"], ROPE), dtype=torch.float64, device="cuda")
        q[:live] = _turn64(big["q"][:live, :, 128:], pos, table, case["interleaved"])
        out["q"] = q
    if case["format"] == "bf16":
        cache = torch.zeros((h["blocks"] * case["block"], E), dtype=torch.float64, device="cuda")
        cache[torch.from_numpy(h["slots"][:live]).to("cuda")] = torch.cat([lat, rope], dim=-1)
        out["cache"] = cache.view(h["blocks"], case["block"], E)
        return out
    group, grid = (32, _grid64(2, 1, 1, 8)) if case["format"] == "fp4" else (64, _grid64(4, 3, 7, 127))
    full = 7.0 if case["format"] == "fp4" else 448.0
    g = lat.reshape(live, DV // group, group)
    k = torch.ceil(torch.log2(g.abs().amax(-1) / full)).clamp(min=-127)
    scale = torch.exp2(k)[..., None]
    mag = g.abs() / scale
    at = torch.searchsorted(grid, mag).clamp(max=len(grid) - 1)
    lo = grid[(at - 1).clamp(min=0)]
    hi = grid[at]
    up = torch.where(mag - lo == hi - mag, at % 2 == 0, mag - lo > hi - mag)
    val = torch.where(up, hi, lo) * torch.sign(g) * scale
    out["rows"] = torch.cat([val.reshape(live, DV), rope], dim=-1)
    return out


def _exact_gather(case, h, seed):
    flat = _big(case, h, seed)["cache"].view(-1, 400)
    bs, slots = case["block"], []
    for r in range(case["batch"]):
        p = np.arange(int(h["cu"][r + 1] - h["cu"][r])) + int(h["starts"][r])
        slots.append(h["table"][r, p // bs].astype(np.int64) * bs + p % bs)
    return _values64(flat[torch.from_numpy(np.concatenate(slots)).to("cuda")])


def _exact_verify(case, h, seed):
    big = _big(case, h, seed)
    tokens = big["tokens"].cpu().numpy()
    paths = np.full((case["batch"], case["nodes"]), -1, dtype=np.int32)
    counts, nexts = [], []
    for r in range(case["batch"]):
        t0, n = int(h["qo"][r]), int(h["qo"][r + 1] - h["qo"][r])
        at, path = 0, [0]
        while True:
            p = big["target"][t0 + at].double().cpu().numpy()
            q = big["draft"][t0 + at].double().cpu().numpy() if case["drawn"] else None
            left, mass, times, chosen = p.copy(), 1.0, 0.0, -1
            for j in range(at + 1, n):
                if int(h["parents"][t0 + j]) != at:
                    continue
                x, u = int(tokens[t0 + j]), float(h["u"][t0 + j])
                if u * mass * (q[x] if case["drawn"] else 1.0) < left[x]:
                    chosen = j
                    break
                if case["drawn"]:
                    times += mass
                    left = np.maximum(p - times * q, 0.0)
                    mass = left.sum()
                else:
                    mass -= left[x]
                    left[x] = 0.0
            if chosen < 0:
                break
            path.append(chosen)
            at = chosen
        paths[r, :len(path)] = path
        counts.append(len(path))
        sums = np.cumsum(left if left.sum() > 0 else p)
        nexts.append(int(np.searchsorted(sums, float(h["u_last"][r]) * sums[-1], side="right")))
    return [torch.from_numpy(np.asarray(v, dtype=np.int32)).to("cuda") for v in (paths, counts, nexts)]


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(one, work(one))
