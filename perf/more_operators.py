"""Cases and plain forms of the operators around a step of rollouts and the scoring of their tokens.

  rotary    pt.rotary              rotary positions of one or several axes on the heads of a fused projection, and the inverse
  drafts    pt.draft_tree          trees of drafted tokens, given by parents: each draft's ancestors and position id
  decode    pt.attn_decode         attention of the trees' tokens over the cached prefix tree (its draft_mask)
  keep      pt.cache_keep          the accepted drafts' keys and values moved together in the cache
  score     pt.token_logprobs      log probabilities of given tokens, with entropy and top alternatives
  grad      pt.token_logprobs_bwd  their gradient

A cache row is a tree node: a prompt shared by the samples below it, or one sample's own continuation. In the flat
layout of a batch a prompt's last row of logits is scored against the first token of each of its completions.
`own` says which of the two forms `run` computes: the plain one in torch operations, or the framework's calls.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the newest token of each of a GRPO batch's 64 completions: 14 q and 2 k heads in front of 2 v heads
        dict(name="rotary, GRPO batch step", op="rotary", T=64, H=16, more=2, D=64, rot=64, axes=1, far=4096, pairs="half", inverse=False, type="bf16"),
        # a long-prompt batch (32 q and 8 k heads) with positions in time, height and width
        dict(name="rotary, long-prompt batch", op="rotary", T=27687, H=40, more=8, D=128, rot=128, axes=3, far=32768, pairs="half", inverse=False, type="bf16"),
        # trees of 8 drafts behind the 64 completions
        dict(name="drafts, GRPO batch", op="drafts", samples=64, q_len=8, shape="wide", lengths=1),
        # a serving loop's step: 4096 requests, up to 64 drafts each
        dict(name="drafts, 4096 requests", op="drafts", samples=4096, q_len=64, shape="any", lengths=2),
        # those 8 drafts attend (14 q heads, 2 kv heads, head_dim 64)
        dict(name="decode, GRPO batch", op="decode", tree="grpo", groups=8, prompt=512, n=8, rmin=64, rmax=256, Hq=14, Hkv=2, D=64, type="bf16", page=16, q_len=8, shape="wide", lengths=3),
        # trees of 32 drafts on every rollout of a long-prompt batch (32 q heads, 8 kv heads, head_dim 128)
        dict(name="decode, long-prompt batch", op="decode", tree="grpo", groups=2, prompt=4096, n=16, rmin=256, rmax=1024, Hq=32, Hkv=8, D=128, type="bf16", page=64, q_len=32, shape="any", lengths=4),
        # what a step of the GRPO batch accepts
        dict(name="keep, GRPO batch", op="keep", samples=64, q_len=8, shape="wide", Hkv=2, D=64, type="bf16", page=16, most=256, lengths=5),
        # the same for 1024 requests with 16 drafts each (8 kv heads, head_dim 128)
        dict(name="keep, 1024 requests", op="keep", samples=1024, q_len=16, shape="any", Hkv=8, D=128, type="bf16", page=16, most=128, lengths=6),
        # a decoding step: 64 samples' chosen tokens, with the entropy and the 20 most likely ones
        dict(name="score, 64 samples", op="score", rows=64, entries="one", V=131072, pad=0, k=20, entropy=True, scale=1.0, type="bf16", lengths=7),
        # the GRPO batch: every flat token under its prefix
        dict(name="score, GRPO batch", op="score", rows=0, entries="tree", V=65536, pad=0, k=0, entropy=True, scale=1.0, type="bf16", lengths=8),
        # documents in fp32, a vocabulary of odd size
        dict(name="grad, documents f32", op="grad", rows=1000, entries="one", V=50001, pad=0, entropy=False, scale=1.0, type="f32", lengths=9),
        # the GRPO batch's policy gradient with an entropy bonus, sampled at temperature 0.8
        dict(name="grad, GRPO batch", op="grad", rows=0, entries="tree", V=65536, pad=0, entropy=True, scale=1.25, type="bf16", lengths=10),
    ]


def _log(rng, a, b):
    return min(b, int(round(a * (b / a) ** rng.random())))


def draw(rng):
    op = rng.choice(["rotary", "drafts", "decode", "decode", "keep", "score", "score", "grad"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    lengths = rng.randrange(1 << 20)
    shape = rng.choice(["any", "wide", "chain"])
    if op == "rotary":
        D = rng.choice([32, 64, 80, 96, 128, 256])
        H = _log(rng, 1, 48)
        T = _log(rng, 1, max(2, min(40000, 27687 * 40 * 256 // (H * D * (2 if kind == "bf16" else 4)))))
        return dict(op=op, T=T, H=H, more=rng.choice([0, 0, 1, 8]), D=D, rot=rng.choice([D, D, D // 2]), axes=rng.choice([1, 1, 2, 3, 4]),
                    far=rng.choice([512, 32768, 1 << 20]), pairs=rng.choice(["half", "half", "near"]), inverse=rng.random() < 0.4, type=kind)
    if op == "drafts":
        return dict(op=op, samples=_log(rng, 1, 4096), q_len=_log(rng, 1, 64), shape=shape, lengths=lengths)
    if op == "keep":
        Hkv, D = rng.choice([(2, 64), (8, 128), (4, 128), (1, 64), (3, 80)])
        q_len, most = _log(rng, 1, 64), _log(rng, 1, 200)
        samples = _log(rng, 1, max(2, min(1024, 100_000_000 // ((q_len + most) * Hkv * D * (2 if kind == "bf16" else 4)))))
        return dict(op=op, samples=samples, q_len=q_len, shape=shape, Hkv=Hkv, D=D, type=kind, page=rng.choice([1, 16, 16, 32, 24]), most=most, lengths=lengths)
    if op == "decode":
        kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hkv, g, D = rng.choice([(2, 7, 64), (8, 4, 128), (4, 4, 128), (2, 4, 256), (1, 8, 64), (8, 1, 128), (2, 6, 96)] if kind == "bf16" else [(2, 1, 32), (2, 3, 64), (4, 2, 128)])
        while True:
            q_len = _log(rng, 1, 64)
            tree = rng.choice(["grpo", "grpo", "docs"])
            if tree == "grpo":
                c = dict(groups=_log(rng, 1, 16), prompt=rng.choice([0, _log(rng, 1, 8192), _log(rng, 64, 8192)]), n=_log(rng, 1, 64))
                c["rmin"] = _log(rng, q_len, 512)
                c["rmax"] = c["rmin"] + _log(rng, 1, 512)
            else:
                c = dict(total=_log(rng, 64, 16384), dmin=q_len, dmax=q_len + _log(rng, 64, 2048))
            case = dict(op=op, tree=tree, **c, Hq=Hkv * g, Hkv=Hkv, D=D, type=kind, page=rng.choice([16, 16, 32, 64]), q_len=q_len, shape=shape, lengths=lengths)
            lens, paths = _tree(case)
            # no more than the listed cases' keys and values, and scores of the plain form
            if sum(lens) * Hkv * D * (2 if kind == "bf16" else 4) <= 8e7 and sum(lens) * len(paths) * Hkv * g * q_len <= 6e8:
                return case
    V = _log(rng, 2, 131072)
    entries = rng.choice(["one", "one", "some", "tree"])
    rows = 0 if entries == "tree" else _log(rng, 1, 8192)
    case = dict(op=op, rows=rows, entries=entries, V=V, pad=rng.choice([0, 0, 1, 63]), entropy=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 1.25, 0.7]), type=kind, lengths=lengths)
    if op == "score":
        case["k"] = min(V, rng.choice([0, 0, 1, 5, 20, 64]))
    limit = 900_000_000 // (2 if kind == "f32" else 1)
    if entries == "tree":
        case["V"] = min(V, 30000)
    elif rows * V > limit:
        case["rows"] = limit // V
    return case


def _tree(case):
    """The tree of a case, the same for every seed: node lengths and root-to-leaf paths."""
    r = random.Random(case["lengths"])
    lens, paths = [], []
    if case["tree"] == "docs":
        left = case["total"]
        while left > 0:
            d = max(case["dmin"], min(left, r.randint(case["dmin"], case["dmax"])))
            paths.append([len(lens)])
            lens.append(d)
            left -= d
        return lens, paths
    for _ in range(case["groups"]):
        root = len(lens)
        lens.append(case["prompt"])
        for _ in range(case["n"]):
            paths.append([root, len(lens)])
            lens.append(r.randint(case["rmin"], case["rmax"]))
    return lens, paths


def _parents(g, n, q_len, shape):
    """Parents [n, q_len] of trees whose drafts come parents first; -1: the last token before the drafts."""
    j = np.arange(q_len)
    if shape == "chain":
        return np.tile(j - 1, (n, 1)).astype(np.int32)
    if shape == "wide":  # every draft has up to four children, in breadth-first order
        up = (j - 1) // 4
        up = np.where(j < 3, -1, np.minimum(up, j - 1))
        return np.tile(up, (n, 1)).astype(np.int32)
    return g.integers(-1, np.maximum(j, 1), (n, q_len)).astype(np.int32) * (j > 0) - (j == 0)


def _counts(g, n, q_len):
    """Drafts of each sample: most of them all, the others any number."""
    return np.where(g.random(n) < 0.75, q_len, g.integers(0, q_len + 1, n)).astype(np.int32)


def _sees(parents):
    """Which draft [.., j] sees which draft [.., i]: itself and those above it."""
    n, q = parents.shape
    sees = np.zeros((n, q, q), bool)
    for j in range(q):
        up = parents[:, j]
        sees[:, j] = np.where(up[:, None] >= 0, sees[np.arange(n), np.maximum(up, 0)], False)
        sees[:, j, j] = True
    return sees


def _words(sees):
    """The same as bits of 32-bit words."""
    n, q, _ = sees.shape
    w = -(-q // 32)
    bits = np.zeros((n, q, w * 32), np.uint64)
    bits[:, :, :q] = sees
    return (bits.reshape(n, q, w, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32).reshape(n * q, w)


def _kept(g, parents, counts):
    """One accepted path of each tree, parents first, then -1."""
    n, q = parents.shape
    kept = np.full((n, q), -1, np.int32)
    for s in range(n):
        path, j = [], int(g.integers(0, counts[s])) if counts[s] else -1
        while j >= 0:
            path.append(j)
            j = int(parents[s, j])
        kept[s, :len(path)] = path[::-1]
    return kept


def _score_tree(case):
    return _tree(dict(tree="grpo", groups=8, prompt=512, n=8, rmin=64, rmax=256, lengths=case["lengths"]))


def _entries(case):
    """(tokens, row_ptr, index): the tokens scored by each row of logits, the same for every seed; None: token i by row i."""
    if case["entries"] == "one":
        return case["rows"], None, None
    if case["entries"] == "some":  # from none to five a row, in order
        per = np.random.default_rng(case["lengths"]).integers(0, 6, case["rows"])
        return int(per.sum()), np.concatenate([[0], per.cumsum()]), None
    lens, paths = _score_tree(case)
    off = np.cumsum([0] + lens)
    T = int(off[-1])
    before = np.arange(T) - 1  # the flat token in front of each; a node's first token follows its parent's last
    before[off[:-1][np.array(lens) > 0]] = -1
    for path in paths:
        for a, b in zip(path, path[1:]):
            before[off[b]] = off[a + 1] - 1
    index = np.argsort(np.where(before < 0, T, before), kind="stable")
    return T, np.concatenate([[0], np.cumsum(np.bincount(before[before >= 0], minlength=T))]), index


# ---------------------------------------------------------------------------------------------------------------
# inputs

def _paged(g, rng, lens, ps, Hkv, D, t):
    """(tables, Kc, Vc) of rows of these lengths."""
    pages = -(-np.array(lens) // ps)
    n_pages = int(pages.sum()) + 3
    width = int(max(1, pages.max()))
    tables = np.full((len(lens), width), -1, np.int32)
    tables[np.arange(width) < pages[:, None]] = rng.permutation(n_pages)[:pages.sum()]
    Kc = torch.randn(n_pages, Hkv, ps, D, device="cuda", generator=g, dtype=t)
    Vc = torch.randn(n_pages, Hkv, ps, D, device="cuda", generator=g, dtype=t)
    return tables, Kc, Vc


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    cuda = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)  # noqa: E731
    t = TYPES[case.get("type", "bf16")]
    op = case["op"]
    if op == "rotary":
        half = case["rot"] // 2
        axes = case["axes"]
        cut = [half * i // axes for i in range(axes + 1)]
        base = 10000.0 if case["far"] < 100000 else 1000000.0
        x = torch.randn(case["T"], case["H"] + case["more"], case["D"], device="cuda", generator=g, dtype=t)
        pos = torch.randint(0, case["far"], (axes, case["T"]), device="cuda", generator=g)
        return dict(op=op, X=x[:, :case["H"]], pos=pos if axes > 1 else pos[0], sections=[b - a for a, b in zip(cut, cut[1:])] if axes > 1 else None,
                    inv_freq=cuda(base ** (-np.arange(half) / half), torch.float32), near=case["pairs"] == "near", inverse=case["inverse"])
    fixed = np.random.default_rng(case["lengths"])  # structures of a case, the same for every seed
    if op in ("score", "grad"):
        N, row_ptr, index = _entries(case)
        R = case["rows"] or N
        V = case["V"]
        wide = torch.empty(R, V + case["pad"], device="cuda", dtype=t)  # (the projection's columns are padded)
        for i in range(0, R, 4096):
            wide[i:i + 4096] = torch.randn(min(4096, R - i), V + case["pad"], device="cuda", generator=g).mul_(3.0).to(t)
        x = wide[:, :V]
        if V > 4:
            x[:, torch.randperm(V, device="cuda", generator=g)[:max(1, V // 100)]] = -torch.inf  # tokens that may not be chosen
        targets = torch.randint(0, V, (N,), device="cuda", generator=g)
        targets[torch.rand(N, device="cuda", generator=g) < 0.05] = -100  # tokens that are not scored
        if V > 4:
            row = _rows_of(N, row_ptr, R)
            place = np.empty(N, np.int64)
            place[np.arange(N) if index is None else index] = row
            at = x[cuda(np.maximum(place, 0), torch.int64), targets.clamp(min=0)]
            targets = torch.where(torch.isinf(at), -100, targets)  # (a scored token is one that may be chosen)
        s = dict(op=op, logits=x, targets=targets, row_ptr=None if row_ptr is None else cuda(row_ptr, torch.int32), index=None if index is None else cuda(index, torch.int32),
                 scale=case["scale"], entropy=case["entropy"], k=case.get("k", 0), row=None if row_ptr is None else cuda(_rows_of(N, row_ptr, R), torch.int64))
        if op == "grad":
            lse, H = _stats(x, case["scale"])
            s.update(lse=lse, H=H if case["entropy"] else None, dlogp=torch.randn(N, device="cuda", generator=g) / max(N, 1),
                     dH=torch.full((R,), 0.01 / R, device="cuda") * (1 + torch.rand(R, device="cuda", generator=g)) if case["entropy"] else None)
        return s
    q_len = case["q_len"]
    if op == "decode":
        lens, paths = _tree(case)
        S = len(paths)
    else:
        S = case["samples"]
        lens = (fixed.integers(0, case.get("most", 4096) + 1, S) + q_len).tolist()
        paths = [[i] for i in range(S)]
    counts = _counts(rng if op == "drafts" else fixed, S, q_len)
    parents = _parents(rng, S, q_len, case["shape"])
    leaf = np.array([p[-1] for p in paths])
    s = dict(op=op, q_len=q_len, parents=cuda(parents, torch.int32).view(-1), lens=cuda(np.array(lens), torch.int32), count=cuda(counts, torch.int32), leaf=cuda(leaf, torch.int64))
    Hkv = case.get("Hkv", 1)
    Hq = case.get("Hq", Hkv)
    if own:  # what a user's program keeps beside its cache: the tree's plan
        import prefix_tree_block_gb300 as pt

        s["plan"] = pt.decode_plan(len(lens), np.cumsum([0] + [len(p) for p in paths]), np.concatenate([np.array(p) for p in paths]), Hq, Hkv, q_len)
    if op == "drafts":
        s["start"] = cuda(rng.integers(0, 4096, S), torch.int32)
        return s
    ps, D = case["page"], case["D"]
    tables, s["Kc"], s["Vc"] = _paged(g, rng, lens, ps, Hkv, D, t)
    s.update(page=ps, tables=cuda(tables, torch.int32))
    if op == "keep":
        s["kept"] = cuda(_kept(rng, parents, counts), torch.int32)
        return s
    s["Q"] = torch.randn(S * q_len, Hq, D, device="cuda", generator=g, dtype=t)
    s["mask"] = cuda(_words(_sees(parents)), torch.int32)
    on = np.zeros((S, len(lens)), bool)
    on[np.repeat(np.arange(S), [len(p) for p in paths]), np.concatenate([np.array(p) for p in paths])] = True
    s.update(on=cuda(on, torch.bool), tokens=sum(lens), O=torch.zeros(S * q_len, Hq, D, device="cuda", dtype=t), LSE=torch.zeros(Hq, S * q_len, device="cuda"))
    if own:
        s["workspace"] = torch.empty(s["plan"].workspace_bytes(D), dtype=torch.uint8, device="cuda")
    return s


def _rows_of(N, row_ptr, R):
    """The row of logits of each entry, -1 behind the last row's."""
    if row_ptr is None:
        return np.arange(N)
    return np.concatenate([np.repeat(np.arange(R), np.diff(row_ptr)), np.full(N - int(row_ptr[-1]), -1)])


def _stats(x, scale):
    """Log-sum-exp and entropy of the rows, in 64 bits, rounded."""
    lse, H = [], []
    for part in x.split(1024):
        z = part.double() * scale
        top = z.amax(1, keepdim=True)
        d = z - top
        e = d.exp()
        total = e.sum(1)
        lse.append((top[:, 0] + total.log()).float())
        H.append((total.log() - torch.where(e > 0, e * d, 0.0).sum(1) / total).float())
    return torch.cat(lse), torch.cat(H)


# ---------------------------------------------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        import prefix_tree_block_gb300 as pt

        if s["op"] == "rotary":
            return pt.rotary(s["X"], s["pos"], s["inv_freq"], sections=s["sections"], interleaved=s["near"], inverse=s["inverse"])
        if s["op"] == "drafts":
            mask, positions = pt.draft_tree(s["parents"], s["lens"], s["plan"], q_count=s["count"], start=s["start"])
            return dict(mask=mask, positions=positions)
        if s["op"] == "decode":
            O, LSE = pt.attn_decode(s["Q"], s["Kc"], s["Vc"], s["tables"], s["lens"], s["plan"], q_count=s["count"], O=s["O"], LSE=s["LSE"], workspace=s["workspace"], draft_mask=s["mask"])
            return dict(O=O, LSE=LSE)
        if s["op"] == "keep":
            pt.cache_keep(s["kept"], s["Kc"], s["Vc"], s["tables"], s["lens"], s["plan"], q_count=s["count"])
            return dict(Kc=s["Kc"], Vc=s["Vc"])
        if s["op"] == "score":
            logp, lse, H, top, ids = pt.token_logprobs(s["logits"], s["targets"], row_ptr=s["row_ptr"], index=s["index"], top_k=s["k"], entropy=s["entropy"], scale=s["scale"])
            return dict(logp=logp, lse=lse, H=H, top=top, ids=ids)
        return pt.token_logprobs_bwd(s["dlogp"], s["logits"], s["targets"], s["lse"], row_ptr=s["row_ptr"], index=s["index"], dentropy=s["dH"], entropy=s["H"], scale=s["scale"])
    return {"rotary": _rotary, "drafts": _drafts, "decode": _decode, "keep": _keep, "score": _score, "grad": _grad}[s["op"]](s)


def _rotary(s):
    x, half = s["X"].float(), s["inv_freq"].numel()
    pos = s["pos"].double()
    if s["sections"] is not None:  # the axis of each pair
        pos = pos.repeat_interleave(torch.tensor(s["sections"], device=x.device), 0, output_size=half).t()
    else:
        pos = pos[:, None]
    angle = pos * s["inv_freq"].double()
    c, si = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if s["inverse"]:
        si = -si
    y = x.clone()
    if s["near"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * si, b * c + a * si
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * si, b * c + a * si
    return y.to(s["X"].dtype)


def _drafts(s):
    q = s["q_len"]
    up = s["parents"].long().view(-1, q)
    j = torch.arange(q, device=up.device)
    real = j < s["count"][:, None]
    up = torch.cat([torch.where(up < 0, q, up), up.new_full((up.shape[0], 1), q)], 1)  # column q: above all drafts
    sees = torch.zeros(up.shape[0], q + 1, q + 1, dtype=torch.bool, device=up.device)
    sees[:, j, j] = True
    for _ in range(max(1, (q - 1).bit_length())):  # twice the steps up each time
        sees = sees | sees.gather(1, up[:, :, None].expand(-1, -1, q + 1))
        up = up.gather(1, up)
    sees = sees[:, :q, :q] & real[:, :, None]
    width = -(-q // 32)
    bits = torch.zeros(sees.shape[0], q, width * 32, dtype=torch.int64, device=up.device)
    bits[:, :, :q] = sees
    words = (bits.view(-1, q, width, 32) << torch.arange(32, device=up.device)).sum(-1)
    first = (s["start"].long() + s["lens"].long())[s["leaf"]] - s["count"].long()
    positions = torch.where(real, first[:, None] + sees.sum(-1) - 1, 0)
    return dict(mask=(words - (words >> 31 << 32)).int().view(-1, width), positions=positions.view(-1))


def _decode(s):
    lens, q, ps, T = s["lens"].long(), s["q_len"], s["page"], s["tokens"]
    Hq, D = s["Q"].shape[1:]
    S, Hkv = s["leaf"].numel(), s["Kc"].shape[1]
    dev = lens.device
    node = torch.repeat_interleave(torch.arange(lens.numel(), device=dev), lens, output_size=T)
    off = torch.arange(T, device=dev) - (lens.cumsum(0) - lens)[node]
    page, row = s["tables"][node, off // ps].long(), off % ps
    K, V = s["Kc"][page, :, row].float(), s["Vc"][page, :, row].float()  # [T, Hkv, D]
    count = s["count"].long()
    draft = off - (lens[s["leaf"]] - count)[:, None]  # [S, T]: which draft of the sample a token of its leaf is
    mine = node == s["leaf"][:, None]
    words = s["mask"].long().view(S, q, -1)
    at = draft.clamp(0, q - 1)
    bit = words.gather(2, (at // 32)[:, None].expand(-1, q, -1)) >> (at % 32)[:, None] & 1
    keep = s["on"][:, node][:, None] & (~mine | (draft < 0))[:, None] | (mine & (draft >= 0))[:, None] & (bit > 0)  # [S, q, T]
    Q = s["Q"].float().view(S, q, Hkv, Hq // Hkv, D)
    score = torch.einsum("sjhgd,thd->hgsjt", Q, K).mul_(D ** -0.5).masked_fill_(~keep, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    O = torch.einsum("hgsjt,thd->sjhgd", p, V) / total.permute(2, 3, 0, 1, 4).clamp(min=1e-30)
    real = (torch.arange(q, device=dev) < count[:, None]).view(-1)  # the other rows stay as they are
    O = torch.where(real[:, None, None], O.reshape(S * q, Hq, D).to(s["Q"].dtype), s["O"])
    return dict(O=O, LSE=torch.where(real, (top + total.log()).reshape(Hq, S * q), s["LSE"]))


def _keep(s):
    ps, kept = s["page"], s["kept"].long()
    i = torch.arange(kept.shape[1], device=kept.device)
    base = s["lens"].long()[s["leaf"]] - s["count"].long()
    moves = kept >= 0
    row, to = torch.where(moves)
    src, dst = base[row] + kept[row, to], base[row] + i[to]
    t = s["tables"]
    ps_, pd = t[s["leaf"][row], src // ps].long(), t[s["leaf"][row], dst // ps].long()
    for cache in (s["Kc"], s["Vc"]):
        cache[pd, :, dst % ps] = cache[ps_, :, src % ps]
    return dict(Kc=s["Kc"], Vc=s["Vc"])


def _score(s):
    x = s["logits"].float() * s["scale"]
    top = x.amax(1, keepdim=True)
    d = x - top
    e = d.exp()
    total = e.sum(1)
    lse = top[:, 0] + total.log()
    out = dict(lse=lse, H=total.log() - torch.where(e > 0, e * d, 0.0).sum(1) / total if s["entropy"] else None, top=None, ids=None)
    if s["k"]:
        raw, ids = s["logits"].float().sort(dim=1, descending=True, stable=True)
        out.update(top=raw[:, :s["k"]] * s["scale"] - lse[:, None], ids=ids[:, :s["k"]])
    target, row = s["targets"], s["row"]
    if row is None:
        row = torch.arange(target.numel(), device=x.device)
    place = target if s["index"] is None else target[s["index"].long()]
    logp = torch.where((place >= 0) & (row >= 0), x[row, place.clamp(min=0)] - lse[row], 0.0)
    return dict(out, logp=logp if s["index"] is None else torch.zeros_like(logp).index_put((s["index"].long(),), logp))


def _grad(s):
    x, lse = s["logits"].float() * s["scale"], s["lse"]
    R, V = x.shape
    target, row, g = s["targets"], s["row"], s["dlogp"]
    if row is None:
        row = torch.arange(target.numel(), device=x.device)
    if s["index"] is not None:
        target, g = target[s["index"].long()], g[s["index"].long()]
    g = torch.where((target >= 0) & (row >= 0), g, 0.0)
    row, target = row.clamp(min=0), target.clamp(min=0)
    each = torch.zeros(R, device=x.device).index_add(0, row, g)
    logp = x - lse[:, None]
    p = logp.exp()
    d = -p * each[:, None]
    if s["entropy"]:
        d = d - torch.where(p > 0, p * (logp + s["H"][:, None]), 0.0) * s["dH"][:, None]
    d.view(-1).index_add_(0, row * V + target, g)
    return (d * s["scale"]).to(s["logits"].dtype)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the same by the definition in 64 bits

def work(case):
    op, es = case["op"], 2 if case.get("type") == "bf16" else 4
    if op == "rotary":
        return dict(bytes=2 * case["T"] * case["H"] * case["D"] * es + 8 * case["axes"] * case["T"] + 2 * case["rot"], flops=3 * case["T"] * case["H"] * case["rot"])
    if op in ("score", "grad"):
        N, row_ptr, index = _entries(case)
        R, V = case["rows"] or N, case["V"]
        moved = R * V * es + 12 * N + 4 * R + (4 * R if row_ptr is not None else 0) + (4 * N if index is not None else 0)
        if op == "score":
            return dict(bytes=moved + 4 * R * case["entropy"] + 12 * R * case["k"], flops=4 * R * V)
        return dict(bytes=moved + R * V * es + 8 * R * case["entropy"], flops=4 * R * V)
    q = case["q_len"]
    if op == "drafts":
        return dict(bytes=case["samples"] * (16 + q * (4 + 8 + 4 * -(-q // 32))), flops=0)
    row = case["Hkv"] * case["D"] * es
    if op == "keep":  # (accepted paths differ from seed to seed: those of one)
        rng = np.random.default_rng(0)
        kept = _kept(rng, _parents(rng, case["samples"], q, case["shape"]), np.full(case["samples"], q))
        moved = int(((kept >= 0) & (kept != np.arange(q))).sum())
        return dict(bytes=4 * row * moved + case["samples"] * (8 + 4 * q) + 1, flops=0)
    lens, paths = _tree(case)
    kept = sum(sum(lens[i] for i in p) * q for p in paths)
    rows = len(paths) * q
    moved = 2 * sum(lens) * row + 2 * rows * row * case["Hq"] // case["Hkv"] + 4 * rows * (case["Hq"] + -(-q // 32)) + 4 * sum(-(-n // case["page"]) + 1 for n in lens)
    return dict(bytes=moved, flops=4 * case["D"] * case["Hq"] * kept)


def exact(case, seed):
    op = case["op"]
    if op == "drafts":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "rotary":
        x = s["X"].double()
        T, H, D = x.shape
        half = case["rot"] // 2
        pos = s["pos"].view(case["axes"], T)
        y = x.clone()
        first = [half * i // case["axes"] for i in range(case["axes"] + 1)]
        for axis in range(case["axes"]):
            for i in range(first[axis], first[axis + 1]):
                a, b = (2 * i, 2 * i + 1) if case["pairs"] == "near" else (i, i + half)
                turn = torch.polar(torch.ones(T, dtype=torch.float64, device="cuda"), pos[axis].double() * s["inv_freq"][i].double() * (-1 if case["inverse"] else 1))
                z = torch.complex(x[:, :, a], x[:, :, b]) * turn[:, None]
                y[:, :, a], y[:, :, b] = z.real, z.imag
        return y
    if op == "keep":
        out = {}
        lens, counts, kept, tables = (s[n].cpu().numpy() for n in ("lens", "count", "kept", "tables"))
        src, dst = [], []
        for i in range(len(lens)):
            for to, j in enumerate(kept[i][kept[i] >= 0]):
                for where, k in ((src, j), (dst, to)):
                    at = int(lens[i]) - int(counts[i]) + int(k)
                    where.append(int(tables[i, at // case["page"]]) * case["page"] + at % case["page"])
        for name in ("Kc", "Vc"):
            flat = s[name].double().transpose(1, 2).flatten(0, 1)  # [slot, head, D]
            flat[torch.tensor(dst, dtype=torch.int64, device="cuda")] = flat[torch.tensor(src, dtype=torch.int64, device="cuda")]
            out[name] = flat.unflatten(0, (-1, case["page"])).transpose(1, 2).contiguous()
        return out
    if op in ("score", "grad"):
        return _exact_score(case, s)
    Hq, Hkv, D, q, ps = case["Hq"], case["Hkv"], case["D"], case["q_len"], case["page"]
    lens, paths = _tree(case)
    O, LSE = s["O"].double(), s["LSE"].double()
    parents, counts = s["parents"].cpu().numpy().reshape(-1, q), s["count"].cpu().numpy()
    for i, path in enumerate(paths):
        K, V = [], []
        for node in path:
            ids = s["tables"][node, :-(-lens[node] // ps)].long()
            K.append(s["Kc"][ids].transpose(1, 2).flatten(0, 1)[:lens[node]])
            V.append(s["Vc"][ids].transpose(1, 2).flatten(0, 1)[:lens[node]])
        K, V = torch.cat(K).double(), torch.cat(V).double()
        c = int(counts[i])
        base = K.shape[0] - c
        for j in range(c):
            up, k = [], j
            while k >= 0:
                up.append(base + k)
                k = int(parents[i, k])
            sel = torch.cat([torch.arange(base, device="cuda"), torch.tensor(up, device="cuda")])
            qs = s["Q"][i * q + j].double().view(Hkv, Hq // Hkv, D)
            sc = torch.matmul(qs, K[sel].permute(1, 2, 0)) / math.sqrt(D)
            LSE[:, i * q + j] = torch.logsumexp(sc, -1).reshape(Hq)
            O[i * q + j] = torch.matmul(torch.softmax(sc, -1), V[sel].transpose(0, 1)).reshape(Hq, D)
    return dict(O=O, LSE=LSE)


def _exact_score(case, s):
    x, V = s["logits"], case["V"]
    N, row_ptr, index = _entries(case)
    R = case["rows"] or N
    token = np.arange(N) if index is None else index
    ptr = np.arange(N + 1) if row_ptr is None else row_ptr
    targets = s["targets"].cpu().numpy()
    if case["op"] == "score":
        lse, H, top = (torch.empty(R, dtype=torch.float64, device="cuda") for _ in range(3))
        top = torch.empty(R, case["k"], dtype=torch.float64, device="cuda")
        logp = torch.zeros(N, dtype=torch.float64, device="cuda")
    else:
        d = torch.empty(R, V, dtype=torch.float64, device="cuda")
        g = s["dlogp"].double()
    for a in range(0, R, 1024):
        b = min(R, a + 1024)
        z = torch.log_softmax(x[a:b].double() * case["scale"], 1)
        p = z.exp()
        h = -torch.xlogy(p, p).sum(1)
        e = np.arange(ptr[a], ptr[b])  # the rows' entries
        r, t = np.repeat(np.arange(b - a), np.diff(ptr[a:b + 1])), token[e]
        r, t = r[targets[t] >= 0], t[targets[t] >= 0]
        r, t, v = (torch.from_numpy(np.ascontiguousarray(u)).cuda() for u in (r, t, targets[t]))
        if case["op"] == "score":
            lse[a:b] = torch.logsumexp(x[a:b].double() * case["scale"], 1)
            H[a:b] = h
            logp[t] = z[r, v]
            if case["k"]:
                top[a:b] = z.topk(case["k"], 1).values
        else:
            each = torch.zeros(b - a, dtype=torch.float64, device="cuda").index_add_(0, r, g[t])
            y = -p * each[:, None]
            if case["entropy"]:
                y -= s["dH"][a:b, None].double() * torch.where(p > 0, p * (z + h[:, None]), 0.0)
            y.index_put_((r, v), g[t], accumulate=True)
            d[a:b] = y * case["scale"]
    if case["op"] == "grad":
        return d
    return dict(logp=logp, lse=lse, H=H if case["entropy"] else None, top=top if case["k"] else None, ids=None)
