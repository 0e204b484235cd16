"""The operators of a speculative decoding step over the paged latent cache, as cases to measure.

A step with drafted tokens has four parts, and each is an operator here:

  append   the new tokens' rows: per-head query norm, latent norm and rotation in one pass, the rows
           written into their cache pages (mla_rope_append)
  tree     absorbed attention of a tree of drafted tokens over the cache (mla_plan_tree, mla_decode_tree,
           mla_decode_tree_fp8)
  verify   acceptance of the drafted tokens against the target's probabilities, from given random
           numbers (mla_verify_tree)
  pages    the cache afterwards: accepted rows moved together (mla_cache_compact); sequences released
           and forked, full pages shared and the last page copied (mla_pages_resize, mla_pages_fork)

With ``own`` false, ``run`` computes a case in plain torch operations (32 bits; 64 where a decision
lies next to a border); with ``own`` true it calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
PAGE, D_C, D_R, D_N, D_V = 64, 512, 64, 128, 128
D_K, D_Q = D_C + D_R, D_N + D_R
SCALE = 1.0 / math.sqrt(D_Q)
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence, V3 heads: what a decode step pays in latency before attention
        dict(name="append_one", kind="append", N=1, H=128, q_norm=False, interleaved=True, split=False),
        # a speculative step's tokens: 32 sequences of 9 nodes, heads normed one by one, an odd count
        dict(name="append_step", kind="append", N=287, H=64, q_norm=True, interleaved=False, split=True),
        # a prefill chunk at V3 geometry
        dict(name="append_chunk", kind="append", N=4096, H=128, q_norm=False, interleaved=True, split=False),
        # V2-Lite geometry, one sequence, a small tree: the smallest attention call
        dict(name="tree_small", kind="tree", H=16, B=1, lo=512, hi=512, T=8, fp8=False),
        # a V3 serving batch with trees of 16 nodes over ragged contexts
        dict(name="tree_batch", kind="tree", H=128, B=32, lo=1000, hi=6000, T=16, fp8=False),
        # one long context, a short tree: the work is split over the cache
        dict(name="tree_long", kind="tree", H=128, B=1, lo=131072, hi=131072, T=5, fp8=False),
        # FP8 rows, padded trees of up to 11 nodes, some sequences with fewer
        dict(name="tree_fp8", kind="tree", H=128, B=24, lo=256, hi=4096, T=11, fp8=True),
        # one sequence, a chain of 4 drafted tokens, bf16 probabilities
        dict(name="verify_one", kind="verify", B=1, T=5, V=32000, bf16=True, draft=True, tree=False),
        # a serving batch's chains against a large vocabulary
        dict(name="verify_batch", kind="verify", B=64, T=6, V=129280, bf16=False, draft=True, tree=False),
        # trees whose drafts carry no probabilities (the likeliest tokens of a drafter), odd vocabulary
        dict(name="verify_tree", kind="verify", B=48, T=24, V=50257, bf16=False, draft=False, tree=True),
        # accepted rows of 256 sequences moved together
        dict(name="compact", kind="compact", B=256, lo=100, hi=900, T=48),
        # half of a beam's sequences released and forked anew from the other half
        dict(name="fork", kind="fork", B=96, lo=200, hi=2000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "append", "tree", "tree", "tree", "verify", "verify", "compact", "fork"])
    if kind == "append":
        return dict(kind=kind, N=_log(rng, 1, 4000), H=rng.choice([8, 16, 32, 64, 128]), q_norm=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, split=rng.random() < 0.5)
    if kind == "tree":
        H, hi = rng.choice([8, 16, 32, 64, 128]), _log(rng, 300, 6000)
        lo = _log(rng, 64, hi)
        return dict(kind=kind, H=H, B=_log(rng, 1, 24), lo=lo, hi=hi, T=_log(rng, 1, 16 if H == 128 else 24),
                    fp8=rng.random() < 0.3)
    if kind == "verify":
        tree = rng.random() < 0.5
        return dict(kind=kind, B=_log(rng, 1, 48), T=rng.randint(2, 24 if tree else 8), V=_log(rng, 1000, 129000),
                    bf16=rng.random() < 0.3, draft=rng.random() < 0.6, tree=tree)
    if kind == "compact":
        lo = _log(rng, 64, 600)
        return dict(kind=kind, B=_log(rng, 1, 256), lo=lo, hi=lo + rng.randint(1, 500), T=rng.randint(2, 64))
    lo = _log(rng, 65, 1500)
    return dict(kind=kind, B=2 * _log(rng, 1, 48), lo=lo, hi=lo + rng.randint(1, 600))


# ------------------------------------------------------------------------- layouts that go by the case
def _lens(case):
    """Lengths (log-uniform, the nodes included) and node counts of a batch: the same for every seed."""
    r = random.Random(case["B"] * 1009 + case["hi"])
    B, T = case["B"], case.get("T", 0)
    lens = [_log(r, case["lo"], case["hi"]) for _ in range(B)]
    nodes = [T if b == 0 or r.random() < 0.7 else r.randint(1, T) for b in range(B)] if T else [0] * B
    lens = [max(s, n + 1) for s, n in zip(lens, nodes)]
    return np.array(lens, dtype=np.int32), np.array(nodes, dtype=np.int32)


def _accepted(case):
    """Accepted nodes of each sequence of a compaction (the root counted): the same for every seed."""
    r = random.Random(case["B"] * 31 + case["T"])
    _, nodes = _lens(case)
    return np.array([r.randint(1, int(n)) for n in nodes], dtype=np.int32)


def _table(lens, spare, rng):
    """Block table over a shuffled pool with `spare` blocks that nobody holds."""
    pages = (lens + PAGE - 1) // PAGE
    nb = int(pages.sum()) + spare
    order = rng.permutation(nb)
    bt = np.full((len(lens), int(pages.max()) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = order[at:at + n]
        at += int(n)
    return bt, nb


def _parents(B, T, tree, rng):
    """Node t's parent: t - 1 in a chain, else a node drawn among those before it, the recent ones likelier."""
    par = np.tile(np.arange(-1, T - 1, dtype=np.int32), (B, 1))
    if tree:
        for t in range(1, T):
            par[:, t] = np.floor((1.0 - rng.random(B) ** 2) * t).astype(np.int32)
    return par


def _ancestors(par):
    """Bit words [B, T, ceil(T / 32)]: bit u of node t's row is set where u is t or an ancestor of t."""
    B, T = par.shape
    see = np.zeros((B, T, 32 * ((T + 31) // 32)), dtype=bool)
    for t in range(T):
        if t:
            see[:, t] = np.take_along_axis(see, np.maximum(par[:, t], 0)[:, None, None], axis=1)[:, 0]
        see[:, t, t] = True
    words = (see.reshape(B, T, -1, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, scale, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# -------------------------------------------------------------------------------------------- prepare
def prepare(case, seed):
    s = globals()["_prepare_" + case["kind"]](case, np.random.default_rng([seed, 17]), _gen(seed))
    s["case"] = case
    if own:
        from mla_latent_cache_gb300 import binding as L
        s["L"] = L
        globals()["_handles_" + case["kind"]](s, L)
    return s


def _prepare_append(case, rng, g):
    N, H = case["N"], case["H"]
    nb = (N + PAGE - 1) // PAGE + 1
    max_pos = 65536
    inv = 10000.0 ** (-torch.arange(0, D_R, 2, dtype=torch.float64, device=DEV) / D_R)
    ang = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * inv
    s = dict(q=_normal(g, (N, H, D_Q), 1.0), kv=_normal(g, (N, D_K), 1.5),
             q_weight=1 + _normal(g, (D_Q,), 0.1) if case["q_norm"] else None, kv_weight=1 + _normal(g, (D_C,), 0.1),
             cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(),
             positions=_dev(rng.integers(0, max_pos, N).astype(np.int32)),
             slots=_dev(rng.permutation(nb * PAGE)[:N].astype(np.int32)),
             q_nope=torch.empty((N, H, D_N), dtype=torch.bfloat16, device=DEV),
             q_pe=torch.empty((N, H, D_R), dtype=torch.bfloat16, device=DEV))
    if case["split"]:
        s["ckv"] = torch.zeros((nb, PAGE, D_C), dtype=torch.bfloat16, device=DEV)
        s["kpe"] = torch.zeros((nb, PAGE, D_R), dtype=torch.bfloat16, device=DEV)
    else:
        s["pool"] = torch.zeros((nb, PAGE, D_K), dtype=torch.bfloat16, device=DEV)
        s["ckv"], s["kpe"] = s["pool"][..., :D_C], s["pool"][..., D_C:]
    return s


def _prepare_tree(case, rng, g):
    lens, nodes = _lens(case)
    B, T, H = case["B"], case["T"], case["H"]
    bt, nb = _table(lens, 1, rng)
    s = dict(q_lat=_normal(g, (B, T, H, D_C), 0.05 if case["fp8"] else 5.0), q_pe=_normal(g, (B, T, H, D_R), 0.1 if case["fp8"] else 5.0),
             block_table=_dev(bt), seq_lens=_dev(lens), node_lens=_dev(nodes), num_blocks=nb,
             mask=_dev(_ancestors(_parents(B, T, True, rng))), max_len=int(lens.max()),
             o_lat=torch.empty((B, T, H, D_C), dtype=torch.bfloat16, device=DEV),
             lse=torch.empty((B, T, H), dtype=torch.float32, device=DEV))
    pool = _normal(g, (nb, PAGE, D_K), 0.1)
    if case["fp8"]:
        lat = pool[..., :D_C].float().view(nb, PAGE, 4, 128)
        sc = lat.abs().amax(-1, keepdim=True) / 448.0
        rows = torch.empty((nb, PAGE, 656), dtype=torch.uint8, device=DEV)
        rows[..., :512] = (lat / sc).to(torch.float8_e4m3fn).view(torch.uint8).reshape(nb, PAGE, 512)
        rows[..., 512:528] = sc.reshape(nb, PAGE, 4).view(torch.uint8)
        rows[..., 528:] = pool[..., D_C:].contiguous().view(torch.uint8)
        s["rows"] = rows
    else:
        s["pool"] = pool
    return s


def _prepare_verify(case, rng, g):
    B, T, V = case["B"], case["T"], case["V"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    par = _parents(B, T, case["tree"], rng)
    width = (V + 7) // 8 * 8   # rows 16-byte aligned
    target = torch.zeros((B, T, width), dtype=dt, device=DEV)
    draft = torch.zeros((B, T, width), dtype=dt, device=DEV)
    logits = torch.randn((B, T, V), generator=g, device=DEV) * 5
    target[..., :V] = torch.softmax(logits, -1)
    q = torch.softmax(logits + 0.7 * torch.randn((B, T, V), generator=g, device=DEV), -1)
    draft[..., :V] = q
    # each child is a draw from its parent's draft distribution
    from_parent = q[torch.arange(B, device=DEV)[:, None], _dev(np.maximum(par, 0)).long()].reshape(B * T, V)
    tokens = torch.multinomial(from_parent, 1, generator=g).view(B, T).int()
    return dict(target=target, draft=draft if case["draft"] else None, tokens=tokens, parents=_dev(par), V=V,
                u_accept=torch.rand((B, T), generator=g, device=DEV), u_sample=torch.rand((B,), generator=g, device=DEV),
                accept_len=torch.empty((B,), dtype=torch.int32, device=DEV),
                accept_idx=torch.empty((B, T), dtype=torch.int32, device=DEV),
                out_tokens=torch.empty((B, T), dtype=torch.int32, device=DEV))


def _prepare_compact(case, rng, g):
    lens, nodes = _lens(case)
    B, T, acc = case["B"], case["T"], _accepted(case)
    bt, nb = _table(lens, 1, rng)
    idx = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        idx[b, :acc[b]] = np.concatenate([[0], 1 + np.sort(rng.choice(nodes[b] - 1, acc[b] - 1, replace=False))]) if acc[b] > 1 else 0
    return dict(pool=_normal(g, (nb, PAGE, D_K), 0.1), block_table=_dev(bt), seq_lens=_dev(lens), node_lens=_dev(nodes),
                accept_len=_dev(acc), accept_idx=_dev(idx), new_lens=torch.empty((B,), dtype=torch.int32, device=DEV))


def _prepare_fork(case, rng, g):
    lens, _ = _lens(case)
    lens += (lens % PAGE == 0).astype(np.int32)   # every sequence has a partly filled page
    B = case["B"]
    bt, nb = _table(lens, B, rng)
    bt = np.concatenate([bt, np.full((B, 1), -1, dtype=np.int32)], 1)
    refs = np.zeros(nb, dtype=np.int32)
    refs[bt[bt >= 0]] = 1
    order = rng.permutation(B)
    src, dst = rng.choice(order[:B // 2], B // 2), order[B // 2:]
    keep = lens.copy()
    keep[dst] = 0
    return dict(pool=_normal(g, (nb, PAGE, D_K), 0.1), block_table=_dev(bt), seq_lens=_dev(lens), keep_lens=_dev(keep),
                refs=_dev(refs), src=_dev(src.astype(np.int32)), dst=_dev(dst.astype(np.int32)),
                fork_status=torch.empty((B // 2,), dtype=torch.int32, device=DEV))


# --------------------------------------------------------------------------- the library's own handles
def _handles_append(s, L):
    s["geom"] = L.make_geom(s["case"]["H"])
    s["cache"] = L.cache_from_split(s["ckv"], s["kpe"])


def _handles_tree(s, L):
    c = s["case"]
    s["geom"] = L.make_geom(c["H"])
    s["batch"] = L.make_batch(c["B"], c["T"], False, s["block_table"].shape[1])
    s["ws_bytes"] = L.mla_workspace_size(s["geom"], s["batch"])
    s["workspace"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    if not c["fp8"]:
        s["cache"] = L.cache_from_pool(s["pool"])


def _handles_verify(s, L):
    s["dtype"] = L.MLA_DTYPE_BF16 if s["case"]["bf16"] else L.MLA_DTYPE_F32


def _handles_compact(s, L):
    s["cache"] = L.cache_from_pool(s["pool"])


def _handles_fork(s, L):
    s["cache"] = L.cache_from_pool(s["pool"])
    s["copies"] = torch.empty((3, s["case"]["B"] // 2), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------------ run
def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["kind"]](s)


def _own_append(s):
    L, c = s["L"], s["case"]
    L.check(L.mla_rope_append(s["geom"], c["N"], s["q"], c["H"] * D_Q, D_Q, s["kv"], D_K, s["q_weight"], s["kv_weight"],
                              EPS, s["cos_sin"], s["cos_sin"].shape[0], s["positions"], c["interleaved"], s["cache"],
                              s["slots"], s["q_nope"], s["q_pe"]), "mla_rope_append")
    return s["q_nope"], s["q_pe"], s["ckv"], s["kpe"]


def _own_tree(s):
    L, c = s["L"], s["case"]
    bt = s["block_table"]
    L.check(L.mla_plan_tree(s["geom"], s["batch"], s["seq_lens"], s["node_lens"], s["workspace"], s["ws_bytes"]),
            "mla_plan_tree")
    if c["fp8"]:
        L.check(L.mla_decode_tree_fp8(s["geom"], s["batch"], s["q_lat"], s["q_pe"], s["rows"], s["num_blocks"], bt,
                                      bt.shape[1], s["seq_lens"], s["node_lens"], s["mask"], 0, s["o_lat"], s["lse"],
                                      s["workspace"], s["ws_bytes"]), "mla_decode_tree_fp8")
    else:
        L.check(L.mla_decode_tree(s["geom"], s["batch"], s["q_lat"], s["q_pe"], s["cache"], bt, bt.shape[1],
                                  s["seq_lens"], s["node_lens"], s["mask"], 0, s["o_lat"], s["lse"], s["workspace"],
                                  s["ws_bytes"]), "mla_decode_tree")
    return s["o_lat"], s["lse"]


def _own_verify(s):
    L, c = s["L"], s["case"]
    L.check(L.mla_verify_tree(c["B"], c["T"], c["V"], s["target"], s["draft"], s["dtype"], s["target"].stride(1),
                              s["tokens"], s["parents"], None, s["u_accept"], s["u_sample"], s["accept_len"],
                              s["accept_idx"], s["out_tokens"]), "mla_verify_tree")
    return s["accept_len"], s["accept_idx"], s["out_tokens"]


def _own_compact(s):
    L, bt = s["L"], s["block_table"]
    L.check(L.mla_cache_compact(s["cache"], bt, bt.shape[1], bt.shape[1], s["seq_lens"], s["node_lens"],
                                s["accept_len"], s["accept_idx"], s["case"]["B"], s["case"]["T"], s["new_lens"]),
            "mla_cache_compact")
    return s["new_lens"], s["pool"]


def _own_fork(s):
    L, bt, B = s["L"], s["block_table"], s["case"]["B"]
    nb = s["pool"].shape[0]
    L.check(L.mla_pages_resize(s["refs"], nb, bt, bt.shape[1], bt.shape[1], s["seq_lens"], s["keep_lens"], B,
                               s["seq_lens"]), "mla_pages_resize")
    L.check(L.mla_pages_fork(s["refs"], nb, bt, bt.shape[1], bt.shape[1], s["seq_lens"], B, s["src"], s["dst"], B // 2,
                             s["copies"]), "mla_pages_fork")
    L.check(L.mla_cache_copy(s["cache"], s["copies"], B // 2), "mla_cache_copy")
    return bt, s["refs"], s["seq_lens"], s["pool"]


def _rotate(x, cs, interleaved):
    """Pairs (2i, 2i + 1), or (i, i + 32), turned by the token's angles: x [..., 64], cs [..., 64] = cos | sin."""
    c, n = cs[..., :32], cs[..., 32:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    a, b = x[..., :32], x[..., 32:]
    return torch.cat([a * c - b * n, a * n + b * c], -1)


def _plain_append(s):
    il = s["case"]["interleaved"]
    q, kv = s["q"].float(), s["kv"].float()
    if s["q_weight"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_weight"].float()
    lat = kv[:, :D_C]
    lat = lat * torch.rsqrt(lat.square().mean(-1, keepdim=True) + EPS) * s["kv_weight"].float()
    cs = s["cos_sin"][s["positions"].long()]
    slot = s["slots"].long()
    s["ckv"][slot // PAGE, slot % PAGE] = lat.bfloat16()
    s["kpe"][slot // PAGE, slot % PAGE] = _rotate(kv[:, D_C:], cs, il).bfloat16()
    return q[..., :D_N].bfloat16(), _rotate(q[..., D_N:], cs[:, None], il).bfloat16(), s["ckv"], s["kpe"]


def _fp8_values(rows):
    """The bf16 values that 656-byte rows stand for in the attention: E4M3(code) x scale, rounded to bf16."""
    lat = rows[..., :512].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    lat = (lat * rows[..., 512:528].contiguous().view(torch.float32).unsqueeze(-1)).flatten(-2).bfloat16()
    return torch.cat([lat, rows[..., 528:].contiguous().view(torch.bfloat16)], -1)


def _plain_tree(s):
    c = s["case"]
    B, T, H, S = c["B"], c["T"], c["H"], s["max_len"]
    j = torch.arange(S, device=DEV)
    blk = s["block_table"].long()[:, j // PAGE].clamp(min=0)
    rows = _fp8_values(s["rows"][blk, j % PAGE]) if c["fp8"] else s["pool"][blk, j % PAGE]
    lens, nodes = s["seq_lens"][:, None].long(), s["node_lens"][:, None].long()
    rows = torch.where((j < lens)[..., None], rows, 0).float()
    node = j - (lens - nodes)                                        # [B, S]: which node a cache row is
    word = s["mask"][:, :, :].gather(2, (node.clamp(0, T - 1) // 32)[:, None].expand(B, T, S))
    bit = (word >> (node.clamp(0, T - 1) % 32)[:, None]) & 1
    t = torch.arange(T, device=DEV)
    see = ((node < 0)[:, None] | (bit == 1)) & (j < lens)[:, None] & (t < nodes)[..., None]     # [B, T, S]
    q = torch.cat([s["q_lat"], s["q_pe"]], -1).float().view(B, T * H, D_K)
    x = (torch.bmm(q, rows.transpose(1, 2)) * SCALE).view(B, T, H, S)
    x = x.masked_fill(~see[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = (x - m).exp()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(B, T * H, S), rows[..., :D_C]).view(B, T, H, D_C) / torch.where(total > 0, total, 1.0)
    return o.bfloat16(), (m + total.log()).squeeze(-1)


def _plain_verify(s):
    # The rule goes through the nodes in their order: a node whose parent is the last accepted one is
    # tested; accepted, it becomes the last accepted one, and the mass left over starts anew.  What is
    # left of p after k rejected draws from q is max(p - C q, 0), C growing by the mass Z each time.
    # Decisions lie next to borders: 64 bits.
    target, draft, tokens, parents, V = s["target"], s["draft"], s["tokens"].long(), s["parents"].long(), s["V"]
    B, T = tokens.shape
    row = torch.arange(B, device=DEV)
    above = parents.clamp(min=0)
    px = target[row[:, None], above, tokens].double()
    qx = draft[row[:, None], above, tokens].double() if draft is not None else None
    u = s["u_accept"].double()
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    C = torch.zeros(B, dtype=torch.float64, device=DEV)
    Z = torch.ones(B, dtype=torch.float64, device=DEV)
    taken = torch.zeros((B, T), dtype=torch.bool, device=DEV)
    taken[:, 0] = True
    refused = torch.zeros((B, T), dtype=torch.bool, device=DEV)   # of the last accepted node's children
    for t in range(1, T):
        asked = parents[:, t] == cur
        if draft is not None:
            left = (px[:, t] - C * qx[:, t]).clamp(min=0)
            yes = asked & (left > 0) & (u[:, t] * qx[:, t] * Z < left)
        else:
            again = (refused & (tokens == tokens[:, t:t + 1])).any(1)
            left = torch.where(again, 0.0, px[:, t])
            yes = asked & (left > 0) & (u[:, t] * Z < left)
        no = asked & ~yes
        taken[:, t] = yes
        refused[:, t] = no
        refused &= ~yes[:, None]
        cur = torch.where(yes, t, cur)
        if draft is not None:
            C = torch.where(yes, 0.0, torch.where(no, C + Z, C))
            Z = torch.where(yes, 1.0, Z)
            if s["case"]["tree"] and t + 1 < T:     # a chain's node has no sibling that would ask for the mass left
                mass = (target[row, cur, :V].double() - C[:, None] * draft[row, cur, :V].double()).clamp(min=0).sum(-1)
                Z = torch.where(no, mass, Z)
        else:
            Z = torch.where(yes, 1.0, torch.where(no, Z - left, Z))
    p = target[row, cur, :V].double()
    if draft is not None:
        left = torch.where(C[:, None] > 0, p - C[:, None] * draft[row, cur, :V].double(), p).clamp(min=0)
    else:
        gone = torch.zeros((B, V + 1), dtype=torch.bool, device=DEV).scatter_(1, torch.where(refused, tokens, V), True)
        left = torch.where(gone[:, :V], 0.0, p)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, p)
    upto = left.cumsum(-1)
    last = V - 1 - (left > 0).flip(-1).int().argmax(-1)
    nxt = torch.minimum((upto <= s["u_sample"].double()[:, None] * upto[:, -1:]).sum(-1), last)
    count = taken.sum(1)
    place = taken.cumsum(1) - 1
    idx = torch.full((B, T + 1), -1, dtype=torch.long, device=DEV)
    idx.scatter_(1, torch.where(taken, place, T), torch.arange(T, device=DEV).expand(B, T))
    out = torch.full((B, T + 1), -1, dtype=torch.long, device=DEV)
    out.scatter_(1, torch.where(taken & (place > 0), place - 1, T), tokens)
    out.scatter_(1, (count - 1)[:, None], nxt[:, None])
    return count.int(), idx[:, :T].int(), out[:, :T].int()


def _plain_compact(s):
    B, T = s["case"]["B"], s["case"]["T"]
    base = (s["seq_lens"] - s["node_lens"]).long()[:, None]
    i = torch.arange(T, device=DEV).expand(B, T)
    kept = i < s["accept_len"][:, None]
    frm = base + torch.where(kept, s["accept_idx"].long(), 0)     # what is not kept moves the root onto itself
    to = base + torch.where(kept, i, 0)
    bt = s["block_table"].long()
    s["pool"][bt.gather(1, to // PAGE), to % PAGE] = s["pool"][bt.gather(1, frm // PAGE), frm % PAGE]
    return (s["seq_lens"] - s["node_lens"] + s["accept_len"]), s["pool"]


def _plain_fork(s):
    bt, refs, lens, pool = s["block_table"], s["refs"], s["seq_lens"], s["pool"]
    page = torch.arange(bt.shape[1], device=DEV)
    held = lambda n: (n[:, None] + PAGE - 1) // PAGE  # noqa: E731
    # release: the pages past the length to keep
    gone = (page >= held(s["keep_lens"])) & (page < held(lens))
    refs.index_add_(0, bt.clamp(min=0).view(-1).long(), -gone.view(-1).int())
    bt.masked_fill_(gone, -1)
    lens.copy_(s["keep_lens"])
    # fork: full pages are shared, the last one is copied into the lowest free block
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src]
    full, tail = n // PAGE, n % PAGE
    free = torch.where(refs == 0, torch.arange(refs.numel(), device=DEV), refs.numel()).sort().values[:len(src)]
    shared = page < full[:, None]
    rows = torch.where(shared, bt[src], -1)
    refs.index_add_(0, rows.clamp(min=0).view(-1).long(), shared.view(-1).int())
    refs.index_add_(0, free, torch.ones_like(free, dtype=torch.int32))
    from_block = bt[src].gather(1, full[:, None].long()).squeeze(1).long()
    rows.scatter_(1, full[:, None].long(), free[:, None].int())
    filled = (torch.arange(PAGE, device=DEV) < tail[:, None])[..., None]
    pool[free] = torch.where(filled, pool[from_block], pool[free])
    bt[dst] = rows
    lens[dst] = n
    return bt, refs, lens, pool


# ----------------------------------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    if kind == "append":
        per_token = case["H"] * D_Q * 2 * 2 + D_K * 2 * 2 + 2 * D_R * 2 + 8
        return {"bytes": case["N"] * per_token + D_C * 2, "flops": case["N"] * (case["H"] * (3 * D_R + 4 * D_Q * case["q_norm"]) + 4 * D_C)}
    if kind == "verify":
        # one row of the target, and one of the drafter, decide the last token of each sequence
        el = 2 if case["bf16"] else 4
        rows = 2 if case["draft"] else 1
        return {"bytes": case["B"] * (rows * case["V"] * el + case["T"] * (12 + 8 + rows * el)), "flops": case["B"] * case["V"] * 3}
    lens, nodes = (x.astype(np.int64) for x in _lens(case))
    if kind == "tree":
        H, T = case["H"], case["T"]
        cached = int(lens.sum()) * (656 if case["fp8"] else 1152)
        queries = int(nodes.sum()) * H
        pairs = int((nodes * (lens - nodes)).sum()) * H
        return {"bytes": cached + queries * (D_K * 2) + case["B"] * T * H * (D_C * 2 + 4), "flops": 2 * pairs * (D_K + D_C)}
    if kind == "compact":
        return {"bytes": int((_accepted(case) - 1).sum()) * 2 * D_K * 2 + case["B"] * (16 + 4 * case["T"]), "flops": 0}
    # the released tables are written, the kept halves' tables read; half a page is copied for each fork
    pages = int(((lens + PAGE - 1) // PAGE).sum())
    return {"bytes": case["B"] // 2 * PAGE * D_K * 2 + 4 * 4 * pages, "flops": 0}


# ---------------------------------------------------------------------------------------------- exact
def exact(case, seed):
    if case["kind"] == "verify":
        return None     # whole numbers: equality says it all
    s = globals()["_prepare_" + case["kind"]](case, np.random.default_rng([seed, 17]), _gen(seed))
    return globals()["_exact_" + case["kind"]](s, case)


def _exact_append(s, case):
    # the rotation as a product of complex numbers
    f = torch.float64
    cs = s["cos_sin"].to(f)[s["positions"].long()]
    turn = torch.complex(cs[:, :32], cs[:, 32:])

    def rot(x):
        if case["interleaved"]:
            return torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous()) * turn.view(-1, *[1] * (x.dim() - 2), 32)).flatten(-2)
        z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous()) * turn.view(-1, *[1] * (x.dim() - 2), 32)
        return torch.cat([z.real, z.imag], -1)

    def norm(x, w):
        return x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.to(f)

    q, kv = s["q"].to(f), s["kv"].to(f)
    if s["q_weight"] is not None:
        q = norm(q, s["q_weight"])
    ckv, kpe = s["ckv"].to(f).clone(), s["kpe"].to(f).clone()
    flat_c, flat_r = ckv.view(-1, D_C), kpe.view(-1, D_R)
    flat_c[s["slots"].long()] = norm(kv[:, :D_C], s["kv_weight"])
    flat_r[s["slots"].long()] = rot(kv[:, D_C:])
    return q[..., :D_N], rot(q[..., D_N:]), ckv, kpe


def _exact_tree(s, case):
    # one sequence and one node at a time, over the rows that the node sees
    B, T, H = case["B"], case["T"], case["H"]
    o = torch.zeros((B, T, H, D_C), dtype=torch.float64, device=DEV)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=DEV)
    lens, nodes = _lens(case)
    bits = s["mask"].cpu().numpy().view(np.uint32)
    for b in range(B):
        S, n = int(lens[b]), int(nodes[b])
        blocks = s["block_table"][b, :(S + PAGE - 1) // PAGE].long()
        rows = (_fp8_values(s["rows"][blocks]) if case["fp8"] else s["pool"][blocks]).reshape(-1, D_K)[:S].double()
        for t in range(n):
            seen = [S - n + u for u in range(n) if (int(bits[b, t, u // 32]) >> (u % 32)) & 1]
            k = torch.cat([rows[:S - n], rows[torch.tensor(seen, dtype=torch.long, device=DEV)]])
            x = (s["q_lat"][b, t].double() @ k[:, :D_C].T + s["q_pe"][b, t].double() @ k[:, D_C:].T) / math.sqrt(D_Q)
            lse[b, t] = torch.logsumexp(x, -1)
            o[b, t] = torch.softmax(x, -1) @ k[:, :D_C]
    return o, lse


def _exact_compact(s, case):
    lens, nodes = _lens(case)
    pool, table, idx = s["pool"].double(), s["block_table"].cpu().numpy(), s["accept_idx"].cpu().numpy()
    flat, was = pool.view(-1, D_K), s["pool"].view(-1, D_K)
    to, frm = [], []
    for b, acc in enumerate(_accepted(case)):
        for i in range(int(acc)):
            for at, rows in ((int(lens[b] - nodes[b]) + i, to), (int(lens[b] - nodes[b]) + int(idx[b, i]), frm)):
                rows.append(int(table[b, at // PAGE]) * PAGE + at % PAGE)
    flat[torch.tensor(to, device=DEV)] = was[torch.tensor(frm, device=DEV)].double()
    return None, pool


def _exact_fork(s, case):
    lens, keep = s["seq_lens"].cpu().numpy(), s["keep_lens"].cpu().numpy()
    table, pool = s["block_table"].cpu().numpy(), s["pool"].double()
    used = {int(table[b, p]) for b in range(case["B"]) if keep[b] for p in range((int(lens[b]) + PAGE - 1) // PAGE)}
    free = iter(x for x in range(pool.shape[0]) if x not in used)
    for b in s["src"].cpu().tolist():
        full, tail, new = int(lens[b]) // PAGE, int(lens[b]) % PAGE, next(free)
        pool[new, :tail] = s["pool"][int(table[b, full]), :tail].double()
    return None, None, None, pool
