"""The speculative-decoding step over a paged cache, in plain Python and float64 -- test
infrastructure only.

The definitions, written out: position p of a request is in slot block_table[r, p // block_size] *
block_size + p % block_size, -1 for a token without a place; blocks are counted by rounding lengths
up; a cache row is 512 latent + 64 rope values, and every head attends to the rows themselves; a
drafted node sees the context, itself and its ancestors.
"""
import numpy as np

from .absorbed import _f64

LORA = 512


def update_block_table(seq, new, table, held, stack, block_size, capacity, num_tokens):
    """Returns (qo_indptr, kv_lens, slots, table, held, stack, short) for lists of lengths,
    table [B, M], held [B] and the stack of free blocks (last = next to be taken).  Entries of a row
    behind those in use may hold anything; a request that is not served names no block in those that
    it would have needed."""
    table, held, stack = np.array(table, dtype=np.int64), list(map(int, held)), list(map(int, stack))
    batch, width = table.shape
    want = [-(-(int(seq[r]) + int(new[r])) // block_size) for r in range(batch)]
    give = [(r, j) for r in range(batch) if want[r] < held[r] for j in range(want[r], held[r])]
    for r, j in reversed(give):          # the first block given back is the next one taken
        assert len(stack) < capacity
        stack.append(int(table[r, j]))
        table[r, j] = -1
    for r in range(batch):
        held[r] = min(held[r], want[r])
    left, short = len(stack), False
    for r in range(batch):
        need = want[r] - held[r]
        if need <= 0:
            continue
        if want[r] > width:
            table[r, held[r]:] = -1
            continue
        left -= need                      # a request that cannot be served leaves none for later ones
        if left < 0:
            short = True
            table[r, held[r]:want[r]] = -1
            continue
        for j in range(held[r], want[r]):
            table[r, j] = stack.pop()
        held[r] = want[r]
    qo, slots = [0], []
    for r in range(batch):
        qo.append(qo[-1] + int(new[r]))
        for i in range(int(new[r])):
            p = int(seq[r]) + i
            blk = int(table[r, p // block_size]) if p // block_size < held[r] else -1
            slots.append(blk * block_size + p % block_size if blk >= 0 else -1)
    slots = (slots + [-1] * num_tokens)[:num_tokens]
    return (np.array(qo), np.array([int(a) + int(b) for a, b in zip(seq, new)]), np.array(slots, dtype=np.int64),
            table, np.array(held), stack, short)


def tree_visibility(parents):
    """parents of one tree -> (bool [n, n]: node i sees node j, depths [n])."""
    n = len(parents)
    seen, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = int(parents[j])
        depth[i] = seen[i].sum() - 1
    return seen, depth


def pack_bits(seen, words):
    """bool [n, m] -> int64 [n, words], bit j % 64 of word j // 64."""
    out = np.zeros((seen.shape[0], words), dtype=np.uint64)
    for i, j in zip(*np.nonzero(seen)):
        out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def tree_attention(q_abs, kv, seen, *, sm_scale, logits_soft_cap=0.0):
    """One request: q_abs [n, H, 576], kv [L, 576] (cache rows, the nodes' own at the end),
    seen bool [n, n] among the nodes (None: a chain).  Node j is key L - n + j; keys before
    the nodes are seen by all.  Returns (o_lat [n, H, 512], lse [n, H]); a row without a key
    has o_lat = 0, LSE = -inf."""
    q, c = _f64(q_abs), _f64(kv)
    n, heads, length = q.shape[0], q.shape[1], c.shape[0]
    o, lse = np.zeros((n, heads, LORA)), np.full((n, heads), -np.inf)
    for i in range(n):
        keys = [k for k in range(length)
                if k < length - n or (seen[i, k - (length - n)] if seen is not None else k - (length - n) <= i)]
        if not keys:
            continue
        x = sm_scale * (q[i] @ c[keys].T)
        if logits_soft_cap > 0:
            x = logits_soft_cap * np.tanh(x / logits_soft_cap)
        m = x.max(axis=1, keepdims=True)
        e = np.exp(x - m)
        tot = e.sum(axis=1, keepdims=True)
        o[i] = (e / tot) @ c[keys][:, :LORA]
        lse[i] = (m + np.log(tot))[:, 0]
    return o, lse


def tree_commit(cache, table, seq, paths, counts):
    """cache [L, NB, BS, E] -> a copy in which accepted node i's row sits at position seq + i."""
    out = cache.copy()
    bs = cache.shape[2]
    for r in range(len(seq)):
        for i in range(int(counts[r])):
            a, b = int(seq[r]) + int(paths[r][i]), int(seq[r]) + i
            out[:, table[r][b // bs], b % bs] = cache[:, table[r][a // bs], a % bs]
    return out
