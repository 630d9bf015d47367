"""Plain statements of the serving operators in 64 bits (numpy), for their tests.

Nothing here is shared with the library: sampled tree acceptance, the page pool and its
copies, and latent attention in its expanded form, each one element at a time.
"""
import numpy as np


# ---- sampled acceptance ----------------------------------------------------------------
def weights(x, temperature):
    """Unnormalised weights of one row of logits (float64)."""
    x = np.asarray(x, np.float64)
    if temperature == 0:
        w = np.zeros(len(x))
        w[int(np.argmax(x))] = 1.0
        return w
    return np.exp((x - x.max()) / float(temperature))


def accept_steps(w, children, g=None):
    """The tests of one node as probabilities, without uniform numbers.

    w: the target's weights; children: the tokens in index order; g: the drafter's
    distribution or None.  Yields (token, the largest u that accepts it, residual weights if
    it is refused)."""
    w = np.array(w, np.float64)
    G = 1.0
    if g is not None:
        g = np.array(g, np.float64)
    for x in children:
        W = w.sum()
        if g is None:
            limit = w[x] / W
            w[x] = 0.0
        else:
            if G <= 0:
                return
            gx = g[x]
            limit = (w[x] * G) / (gx * W) if gx * W > 0 else (np.inf if w[x] > 0 else 0.0)
            w = np.maximum(w - g * (W / G), 0.0)
            G -= gx
            g[x] = w[x] = 0.0
        yield x, limit, w.copy()


def sample_tree(logits, parent, tokens, uniforms, temperature, draft=None, by_node=False):
    """accept_len, path, new_tokens of one sequence (logits [Q, V] float64)."""
    Q, V = logits.shape
    path, emit = np.full(Q, -1, np.int32), np.full(Q, -1, np.int32)
    path[0] = 0
    node, count = 0, 0
    while True:
        if np.isnan(logits[node]).any() or not np.isfinite(logits[node].max()):
            return count, path, emit
        w = weights(logits[node], temperature)
        kids = [i for i in range(node + 1, Q)
                if parent[i] == node and 0 <= tokens[i] < V]
        if temperature == 0:
            top = int(np.argmax(w))
            nxt = next((i for i in kids if tokens[i] == top), None)
        else:
            g = None
            if draft is not None:
                row = node if by_node else count
                g = draft[row] if row < len(draft) else None
                if g is None:
                    kids = []
            nxt = None
            for i, (x, limit, left) in zip(kids, accept_steps(w, tokens[kids], g)):
                if float(uniforms[i]) < limit or left.sum() == 0:
                    nxt = i
                    break
                w = left
        if nxt is None:
            total = np.cumsum(w)
            emit[count] = int(np.searchsorted(total, float(uniforms[0]) * total[-1],
                                              side="right"))
            return count, path, emit
        emit[count] = tokens[nxt]
        count += 1
        path[count] = nxt
        node = nxt


# ---- the page pool -----------------------------------------------------------------------
class Pool:
    """A page pool as lists of Python integers."""

    def __init__(self, rows, max_pages, num_pages, page_size):
        self.table = np.full((rows, max_pages), -1, np.int32)
        self.n = np.zeros(rows, np.int32)
        self.ref = np.zeros(num_pages, np.int32)
        self.ps = page_size

    def pages_of(self, keys):
        return -(-int(keys) // self.ps)

    def reserve(self, length, new_length):
        """The copy list, or None (and no change) when pages run out."""
        want = {}
        for r in range(len(self.n)):
            if new_length[r] > length[r]:
                for k in range(length[r] // self.ps,
                               min(int(self.n[r]), self.pages_of(new_length[r]))):
                    if self.ref[self.table[r, k]] > 1:
                        want.setdefault(int(self.table[r, k]), []).append(r)
        keeper = {p: rs[0] for p, rs in want.items() if len(rs) == self.ref[p]}
        copies = np.full((len(self.n), 3), -1, np.int32)
        copies[:, 2] = 0
        free = np.flatnonzero(self.ref == 0).tolist()
        table, n, ref = self.table.copy(), self.n.copy(), self.ref.copy()
        for r in range(len(n)):
            if new_length[r] <= length[r]:
                continue
            for k in range(length[r] // self.ps, self.pages_of(new_length[r])):
                old = int(table[r, k]) if k < n[r] else -1
                if old >= 0 and (self.ref[old] == 1 or keeper.get(old) == r):
                    continue
                if not free:
                    return None
                new = free.pop(0)
                ref[new] = 1
                table[r, k] = new
                if old >= 0:
                    ref[old] -= 1
                    if k == length[r] // self.ps and length[r] % self.ps:
                        copies[r] = (old, new, length[r] % self.ps)
            n[r] = max(int(n[r]), self.pages_of(new_length[r]))
        self.table, self.n, self.ref = table, n, ref
        return copies

    def fork(self, fork_from, length):
        for r, s in enumerate(fork_from):
            if s >= 0:
                k = self.pages_of(length[r])
                self.table[r, :k] = self.table[s, :k]
                np.add.at(self.ref, self.table[s, :k], 1)
                self.n[r] = k

    def release(self, keep):
        for r, keys in enumerate(keep):
            if keys >= 0:
                for k in range(self.pages_of(keys), int(self.n[r])):
                    self.ref[self.table[r, k]] -= 1
                    self.table[r, k] = -1
                self.n[r] = min(int(self.n[r]), self.pages_of(keys))

    def compact(self):
        used = int((self.ref > 0).sum())
        src = [p for p in range(used, len(self.ref)) if self.ref[p] > 0]
        dst = [p for p in range(used) if self.ref[p] == 0]
        to = dict(zip(src, dst))
        for r in range(len(self.n)):
            for k in range(int(self.n[r])):
                self.table[r, k] = to.get(int(self.table[r, k]), self.table[r, k])
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        return np.array([(a, b, self.ps) for a, b in to.items()], np.int32).reshape(-1, 3)

    def check(self):
        """The counts are those of the tables."""
        count = np.zeros_like(self.ref)
        for r in range(len(self.n)):
            np.add.at(count, self.table[r, :self.n[r]], 1)
            assert (self.table[r, self.n[r]:] == -1).all()
        assert np.array_equal(count, self.ref)


def copy_pages(cache, page_size, copies):
    """cache [layers, rows, d] changed in place."""
    for s, d, n in copies:
        if s >= 0:
            cache[:, d * page_size:d * page_size + n] = cache[:, s * page_size:s * page_size + n]


# ---- latent attention, expanded form -------------------------------------------------------
def prefill(q_nope, q_pe, w_kv, keys, rope_keys, prefix, scale):
    """One sequence: q_nope [n,H,dn], q_pe [n,H,dr], w_kv [H,dn+dv,dl], keys [m,dl],
    rope_keys [m,dr] (float64) -> [n,H,dv]; query i sees keys 0 .. prefix + i."""
    n, H, dn = q_nope.shape
    out = np.zeros((n, H, w_kv.shape[1] - dn))
    hidden = np.arange(len(keys))[None] > prefix + np.arange(n)[:, None]
    for h in range(H):
        kv = keys @ w_kv[h].T
        s = (q_nope[:, h] @ kv[:, :dn].T + q_pe[:, h] @ rope_keys.T) * scale
        s[hidden] = -np.inf
        p = np.exp(s - s.max(1, keepdims=True))
        out[:, h] = (p / p.sum(1, keepdims=True)) @ kv[:, dn:]
    return out
