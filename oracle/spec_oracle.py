"""Float64 CPU oracle for the speculative decoding step over the paged latent cache.

TEST INFRASTRUCTURE ONLY, like ``mla_oracle``: plain definitions in float64 NumPy, no
code shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# Row append: norms, rotation
# ---------------------------------------------------------------------------
def rms_norm_ref(x: np.ndarray, weight, eps: float) -> np.ndarray:
    """x / sqrt(mean(x^2) + eps) * weight over the last axis; weight None leaves x as it is."""
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight


def rotate_ref(x: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """Pairs (2k, 2k+1), or (k, k+32), of the last 64 values as complex numbers times e^{i angle}.

    ``cos_sin`` [..., 64] (cos | sin) broadcasts against x [..., 64].
    """
    turn = cos_sin[..., :32] + 1j * cos_sin[..., 32:]
    z = (x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :32] + 1j * x[..., 32:]) * turn
    out = np.empty(z.shape[:-1] + (64,))
    if interleaved:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    else:
        out[..., :32], out[..., 32:] = z.real, z.imag
    return out


def rope_append_ref(q, kv, q_weight, kv_weight, eps, cos_sin, positions, interleaved):
    """(q_nope [N,H,128], q_pe [N,H,64], rows [N,576]) of N new tokens; q [N,H,192], kv [N,576]."""
    cs = cos_sin[positions]
    q = rms_norm_ref(q, q_weight, eps)
    rows = np.concatenate([rms_norm_ref(kv[:, :512], kv_weight, eps), rotate_ref(kv[:, 512:], cs, interleaved)], -1)
    return q[..., :128], rotate_ref(q[..., 128:], cs[:, None], interleaved), rows


# ---------------------------------------------------------------------------
# Verification of drafted tokens
# ---------------------------------------------------------------------------
def verify_ref(target, draft, tokens, parents, n, u_accept, u_sample):
    """One sequence: (accepted node indices, next token), by rejection sampling with residuals
    written as normalised distributions: a refused draw x ~ q turns the distribution r into
    max(r - q, 0) normalised.  target [T, V]; draft [T, V], or None for point masses.

    The rule's first test is against the row as it is (its mass taken as 1).
    """
    if n == 0:
        return [], -1
    V = target.shape[1]
    mass = lambda x: np.where((x > 0) & (x < np.inf), x, 0.0)  # noqa: E731
    path, cur = [0], 0
    left, Z = mass(target[0]), 1.0      # what is left of cur's row, unnormalised, and its mass
    for t in range(1, n):
        if parents[t] != cur or not (0 <= tokens[t] < V) or not (0 <= parents[t] < t):
            continue
        x = int(tokens[t])
        q = mass(draft[cur]) if draft is not None else np.eye(1, V, x)[0]
        if left[x] > 0 and u_accept[t] * q[x] * Z < left[x]:
            path.append(t)
            cur, left, Z = t, mass(target[t]), 1.0
        elif draft is not None:
            left = np.maximum(left - Z * q, 0.0)
            Z = float(left.sum())
        else:
            Z -= left[x]
            left = left.copy()
            left[x] = 0.0
    if not left.sum() > 0:
        left = mass(target[cur])
    if not left.sum() > 0:
        return path, -1
    upto = np.cumsum(left)
    over = np.nonzero(upto > u_sample * upto[-1])[0]
    return path, int(over[0]) if len(over) else int(np.nonzero(left > 0)[0][-1])


# ---------------------------------------------------------------------------
# Pages
# ---------------------------------------------------------------------------
class Pages:
    """Block table, holders' counts and pool of a paged cache, one page at a time."""

    def __init__(self, block_table, refs, lens, pool=None):
        self.bt, self.refs, self.lens = block_table.copy(), refs.copy(), lens.copy()
        self.pool = None if pool is None else pool.copy()

    def _take(self):
        free = np.nonzero(self.refs == 0)[0]
        if not len(free):
            return None
        self.refs[free[0]] = 1
        return int(free[0])

    def resize(self, new_lens):
        held = [(int(s) + 63) // 64 for s in self.lens]
        for b, s in enumerate(new_lens):
            for p in range((int(s) + 63) // 64, held[b]):
                self.refs[self.bt[b, p]] -= 1
                self.bt[b, p] = -1
        for b, s in enumerate(new_lens):
            self.lens[b] = s
            for p in range(held[b], (int(s) + 63) // 64):
                k = self._take()
                if k is None:
                    self.lens[b] = 64 * p
                    break
                self.bt[b, p] = k

    def fork(self, src, dst):
        """Well-formed forks; returns copies [3, F]."""
        out = np.zeros((3, len(src)), dtype=np.int32)
        refs = self.refs.copy()      # who holds what when the call begins
        for f, (s, d) in enumerate(zip(src, dst)):
            full, tail = divmod(int(self.lens[s]), 64)
            out[:, f] = -1, -1, 0
            if tail and (s != d or refs[self.bt[s, full]] > 1):
                free = np.nonzero((self.refs == 0) & (refs == 0))[0]
                if not len(free):
                    out[0, f] = -2
                    continue
                out[:, f] = self.bt[s, full], free[0], tail
                self.refs[free[0]] = 1
        for f, (s, d) in enumerate(zip(src, dst)):
            if out[0, f] == -2:
                continue
            full = int(self.lens[s]) // 64
            if s == d:
                if out[2, f]:
                    self.refs[out[0, f]] -= 1
                    self.bt[d, full] = out[1, f]
                continue
            self.bt[d] = -1
            self.bt[d, :full] = self.bt[s, :full]
            np.add.at(self.refs, self.bt[s, :full], 1)
            if out[2, f]:
                self.bt[d, full] = out[1, f]
            self.lens[d] = self.lens[s]
        return out

    def copy(self, copies):
        for f, t, n in copies.T:
            if n:
                self.pool[t, :n] = self.pool[f, :n]

    def compact(self, nodes, accept_len, accept_idx):
        """The pool after the move, and the new lengths."""
        was = self.pool.copy()
        for b in range(len(self.lens)):
            base = int(self.lens[b] - nodes[b])
            for i in range(int(accept_len[b])):
                t, f = base + i, base + int(accept_idx[b, i])
                self.pool[self.bt[b, t // 64], t % 64] = was[self.bt[b, f // 64], f % 64]
        return (self.lens - nodes + accept_len).astype(np.int32)

    def check(self):
        """Every count is the number of table entries that hold the block."""
        n = np.zeros_like(self.refs)
        for b, s in enumerate(self.lens):
            np.add.at(n, self.bt[b, :(int(s) + 63) // 64], 1)
        assert np.array_equal(n, self.refs)


# ---------------------------------------------------------------------------
# Attention of a tree of drafted tokens
# ---------------------------------------------------------------------------
def tree_visible(S: int, n: int, see: np.ndarray) -> np.ndarray:
    """Boolean [T, S]: node t < n sees the rows before the last n, and row S - n + u where see[t, u]."""
    T = see.shape[0]
    m = np.zeros((T, S), dtype=bool)
    m[:n, :S - n] = True
    m[:n, S - n:] = see[:n, :n]
    return m


def tree_decode_ref(q_lat, q_pe, pool, block_table, seq_lens, node_lens, see, scale=1.0 / np.sqrt(192.0)):
    """(o_lat [B,T,H,512], lse [B,T,H]); pool [num_blocks, 64, 576], see boolean [B, T, T].

    Only the rows that a node sees take part in its sums.
    """
    B, T, H, _ = q_lat.shape
    o = np.zeros((B, T, H, 512))
    lse = np.full((B, T, H), -np.inf)
    for b in range(B):
        S, n = int(seq_lens[b]), min(int(node_lens[b]), int(seq_lens[b]))
        if S == 0:
            continue
        rows = pool[block_table[b, :(S + 63) // 64]].reshape(-1, 576)[:S]
        vis = tree_visible(S, n, see[b])
        for t in range(n):
            r = rows[vis[t]]
            if not len(r):
                continue
            x = (q_lat[b, t] @ r[:, :512].T + q_pe[b, t] @ r[:, 512:].T) * scale
            m = x.max(-1, keepdims=True)
            p = np.exp(x - m)
            lse[b, t] = (m + np.log(p.sum(-1, keepdims=True)))[:, 0]
            o[b, t] = p @ r[:, :512] / p.sum(-1, keepdims=True)
    return o, lse


def see_words(see: np.ndarray) -> np.ndarray:
    """Boolean [B, T, T] as bit words int32 [B, T, ceil(T / 32)]; spare bits are set (nobody may look at them)."""
    B, T, _ = see.shape
    W = (T + 31) // 32
    bits = np.ones((B, T, 32 * W), dtype=np.uint64)
    bits[..., :T] = see
    return (bits.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def ancestors(parents: np.ndarray) -> np.ndarray:
    """Boolean [B, T, T]: node t sees itself and the nodes above it; parents[b, t] < t."""
    B, T = parents.shape
    see = np.zeros((B, T, T), dtype=bool)
    for b in range(B):
        for t in range(T):
            u = t
            while u >= 0:
                see[b, t, u] = True
                u = int(parents[b, u]) if u else -1
    return see
