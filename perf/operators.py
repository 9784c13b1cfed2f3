"""Cases and plain forms of the rollout-decoding operators: a paged key/value cache for the nodes of a prefix tree,
and the attention of the newest tokens of every sample over it.

  tables   pt.cache_tables    page tables, slots and position ids of one step, from the rows' lengths
  write    pt.cache_write     the step's keys and values into their slots
  decode   pt.attn_decode     attention of each sample's last tokens over its path through the tree

A cache row is a tree node: a prompt shared by the samples below it, or one sample's own continuation.
`own` says which of the two forms `run` computes: the plain one in torch operations, or the framework's calls.
"""
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decoding step of a GRPO batch: 64 completions grow by a token, the 8 prompts stand
        dict(name="tables, GRPO batch step", op="tables", rows=72, page=16, most=768, step=64, prefill=0, release=0, trim=0, pad=0, lengths=1),
        # a serving loop's mixed step: prompts come in, requests step, end, or take back rejected draft tokens
        dict(name="tables, mixed step of 4096 rows", op="tables", rows=4096, page=16, most=4096, step=2200, prefill=400, release=300, trim=300, pad=4099, lengths=2),
        # the newest token of each of the GRPO batch's 64 completions (14 q heads, 2 kv heads, head_dim 64)
        dict(name="write, GRPO batch step", op="write", tree="grpo", groups=8, prompt=512, n=8, rmin=64, rmax=256, Hq=14, Hkv=2, D=64, type="bf16", page=16, whole=False, pad=0, lengths=3),
        # the whole long-prompt GRPO batch put into the cache (32 q heads, 8 kv heads, head_dim 128)
        dict(name="write, long-prompt batch", op="write", tree="grpo", groups=2, prompt=4096, n=16, rmin=256, rmax=1024, Hq=32, Hkv=8, D=128, type="bf16", page=64, whole=True, pad=0, lengths=4),
        # packed documents in fp32, padded to a fixed token count
        dict(name="write, packed documents f32", op="write", tree="docs", total=16384, dmin=64, dmax=2048, Hq=8, Hkv=2, D=256, type="f32", page=32, whole=True, pad=1021, lengths=5),
        # the tiny fp32 GRPO group: a call's own cost
        dict(name="decode, tiny group f32", op="decode", tree="grpo", groups=1, prompt=16, n=4, rmin=8, rmax=8, Hq=2, Hkv=2, D=32, type="f32", page=16, q_len=1, lengths=6),
        # a step of the GRPO batch: latency of a small model
        dict(name="decode, GRPO batch", op="decode", tree="grpo", groups=8, prompt=512, n=8, rmin=64, rmax=256, Hq=14, Hkv=2, D=64, type="bf16", page=16, q_len=1, lengths=7),
        # multi-turn rollouts: root 1024 -> 4 x 512 -> 4 x U[128, 384]
        dict(name="decode, depth-3 tree", op="decode", tree="deep", root=1024, mids=4, mid=512, n=4, rmin=128, rmax=384, Hq=16, Hkv=4, D=128, type="bf16", page=32, q_len=1, lengths=8),
        # a step of the long-prompt GRPO batch
        dict(name="decode, long-prompt batch", op="decode", tree="grpo", groups=2, prompt=4096, n=16, rmin=256, rmax=1024, Hq=32, Hkv=8, D=128, type="bf16", page=64, q_len=1, lengths=9),
        # documents that share nothing, at head_dim 256
        dict(name="decode, documents D=256", op="decode", tree="docs", total=16384, dmin=64, dmax=2048, Hq=8, Hkv=2, D=256, type="bf16", page=64, q_len=1, lengths=10),
        # draft blocks of 16 tokens verified at once on every rollout of a long-prompt batch
        dict(name="decode, 16-token drafts", op="decode", tree="grpo", groups=2, prompt=4096, n=16, rmin=256, rmax=1024, Hq=16, Hkv=4, D=128, type="bf16", page=32, q_len=16, lengths=11),
        # rollouts over prompts of 32768 tokens, 64 to a prompt
        dict(name="decode, 32768-token prompts", op="decode", tree="grpo", groups=2, prompt=32768, n=64, rmin=512, rmax=2048, Hq=32, Hkv=8, D=128, type="bf16", page=64, q_len=1, lengths=12),
    ]


def _log(rng, a, b):
    return min(b, int(round(a * (b / a) ** rng.random())))


def draw(rng):
    op = rng.choice(["tables", "write", "decode", "decode"])
    lengths = rng.randrange(1 << 20)
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "tables":
        rows = _log(rng, 1, 4096)
        part = [rng.random() for _ in range(4)]
        cut = [int(rows * p / (sum(part) + rng.random())) for p in part]
        return dict(op=op, rows=rows, page=page, most=_log(rng, 64, 4096), step=cut[0], prefill=cut[1] // 4, release=cut[2] // 2, trim=cut[3] // 2,
                    pad=rng.choice([0, _log(rng, 1, 5000)]), lengths=lengths)
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind == "bf16":
        Hkv, g, D = rng.choice([(2, 7, 64), (8, 4, 128), (4, 4, 128), (2, 4, 256), (1, 8, 64), (8, 1, 128), (3, 5, 64), (2, 6, 96)])
    else:
        Hkv, g, D = rng.choice([(2, 1, 32), (2, 3, 64), (4, 2, 128), (2, 7, 80)])
    q_len = rng.choice([1, 1, 1, 2, 5, 16]) if op == "decode" else 1
    while True:
        tree = rng.choice(["grpo", "grpo", "deep", "docs"])
        if tree == "grpo":
            shape = dict(groups=_log(rng, 1, 16), prompt=rng.choice([0, _log(rng, 1, 16384), _log(rng, 64, 16384)]), n=_log(rng, 1, 64))
        elif tree == "deep":
            shape = dict(root=_log(rng, 1, 8192), mids=_log(rng, 1, 8), mid=_log(rng, 1, 2048), n=_log(rng, 1, 12))
        else:
            shape = dict(total=_log(rng, 64, 32768), dmin=rng.choice([1, 64]), dmax=_log(rng, 64, 4096))
        if tree != "docs":
            shape["rmin"] = _log(rng, q_len, 512)
            shape["rmax"] = shape["rmin"] + _log(rng, 1, 1024)
        elif shape["dmin"] < q_len:
            shape["dmin"] = q_len
        case = dict(op=op, tree=tree, **shape, Hq=Hkv * g, Hkv=Hkv, D=D, type=kind, page=page, lengths=lengths)
        lens, paths = _tree(case)
        # no more than the largest listed case's keys and values, and scores of the plain form
        if sum(lens) * Hkv * D * (2 if kind == "bf16" else 4) <= 2.5e8 and (op == "write" or sum(lens) * len(paths) * Hkv * g * q_len <= 4e8):
            break
    if op == "write":
        return dict(case, whole=rng.random() < 0.7, pad=rng.choice([0, _log(rng, 1, 2000)]))
    return dict(case, q_len=q_len)


def _tree(case):
    """The tree of a case, the same for every seed: node lengths and root-to-leaf paths."""
    r = random.Random(case["lengths"])
    lens, paths = [], []
    if case["tree"] == "docs":
        left = case["total"]
        while left > 0:
            d = r.randint(case["dmin"], max(case["dmin"], case["dmax"]))
            d = d if left - d < case["dmin"] else min(d, left)
            paths.append([len(lens)])
            lens.append(d)
            left -= d
        return lens, paths
    if case["tree"] == "grpo":
        tops = [[case["prompt"]]] * case["groups"]
    else:
        tops = [[case["root"]] + [case["mid"]] * case["mids"]]
    for top in tops:
        root = len(lens)
        lens.append(top[0])
        for mid in top[1:] or [None]:
            up = [root]
            if mid is not None:
                up.append(len(lens))
                lens.append(mid)
            for _ in range(case["n"]):
                paths.append(up + [len(lens)])
                lens.append(r.randint(case["rmin"], case["rmax"]))
    return lens, paths


def _steps(case):
    """held and added tokens of the rows of a tables case, the same for every seed."""
    g = np.random.default_rng(case["lengths"])
    n, most = case["rows"], case["most"]
    order = g.permutation(n)
    a, b, c, d = case["step"], case["prefill"], case["release"], case["trim"]
    held = g.integers(1, most - 32, n)
    added = np.zeros(n, np.int64)
    added[order[:a]] = 1
    new = order[a:a + b]
    held[new], added[new] = 0, g.integers(1, most + 1, new.size)
    out = order[a + b:a + b + c]
    added[out] = -held[out]
    back = order[a + b + c:a + b + c + d]
    added[back] = -np.minimum(held[back], g.integers(1, 17, back.size))
    return held, added


# ---------------------------------------------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    ps = case["page"]
    if case["op"] == "tables":
        held, added = _steps(case)
        width = -(-case["most"] // ps)
        pages = -(-held // ps)
        grown = np.maximum(-(-(held + added) // ps) - pages, 0).sum()
        cap = int(pages.sum() + grown + 64)  # pages of the pool
        ids = rng.permutation(cap).astype(np.int32)
        tables = np.full((held.size, width), -1, np.int32)
        tables[np.arange(width) < pages[:, None]] = ids[:pages.sum()]
        head = int(rng.integers(0, 4 * cap))  # the free ring has been round several times
        ring = ids[rng.integers(0, max(1, pages.sum()), cap)]
        free = ids[pages.sum():]
        ring[(head + np.arange(free.size)) % cap] = free
        new = int(np.maximum(added, 0).sum()) + case["pad"]
        cuda = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)  # noqa: E731
        return dict(op="tables", page=ps, new=new, held=cuda(held, torch.int32), added=cuda(added, torch.int32), start=cuda(rng.integers(0, 4096, held.size), torch.int32),
                    tables=cuda(tables, torch.int32), ring=cuda(ring, torch.int32), counters=torch.tensor([head, head + free.size], dtype=torch.int64, device="cuda"))
    lens, paths = _tree(case)
    Hq, Hkv, D, t = case["Hq"], case["Hkv"], case["D"], TYPES[case["type"]]
    pages = -(-np.array(lens) // ps)
    n_pages = int(pages.sum()) + 3
    width = int(max(1, pages.max()))
    tables = np.full((len(lens), width), -1, np.int32)
    tables[np.arange(width) < pages[:, None]] = rng.permutation(n_pages)[:pages.sum()]
    Kc = torch.randn(n_pages, Hkv, ps, D, device="cuda", generator=g, dtype=t)
    Vc = torch.randn(n_pages, Hkv, ps, D, device="cuda", generator=g, dtype=t)
    if case["op"] == "write":
        if case["whole"]:
            node = np.repeat(np.arange(len(lens)), lens)
            off = np.arange(sum(lens)) - np.repeat(np.cumsum(lens) - lens, lens)
        else:
            node = np.array([p[-1] for p in paths])
            off = np.array(lens)[node] - 1
        slots = tables[node, off // ps].astype(np.int64) * ps + off % ps
        slots = np.concatenate([slots, np.full(case["pad"], -1, np.int64)])
        # the tokens' keys and values, parts of one projection's output
        qkv = torch.randn(slots.size, Hq + 2 * Hkv, D, device="cuda", generator=g, dtype=t)
        return dict(op="write", page=ps, K=qkv[:, Hq:Hq + Hkv], V=qkv[:, Hq + Hkv:], slots=torch.from_numpy(slots).cuda(), real=slots.size - case["pad"], Kc=Kc, Vc=Vc)
    q_len, S = case["q_len"], len(paths)
    Q = torch.randn(S * q_len, Hq, D, device="cuda", generator=g, dtype=t)
    on = np.zeros((S, len(lens)), bool)
    for s, p in enumerate(paths):
        on[s, p] = True
    leaf = np.array([p[-1] for p in paths])
    state = dict(op="decode", page=ps, q_len=q_len, Q=Q, Kc=Kc, Vc=Vc, tables=torch.from_numpy(tables).cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 on=torch.from_numpy(on).cuda(), leaf=torch.from_numpy(leaf).cuda(), tokens=sum(lens), paths=paths)
    if own:  # what a user's program keeps beside its cache: the tree's plan and the scratch
        import prefix_tree_block_gb300 as pt

        ptr = np.cumsum([0] + [len(p) for p in paths])
        plan = pt.decode_plan(len(lens), ptr, np.concatenate([np.array(p) for p in paths]), Hq, Hkv, q_len)
        state.update(plan=plan, workspace=torch.empty(plan.workspace_bytes(D), dtype=torch.uint8, device="cuda"))
    return state


# ---------------------------------------------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        import prefix_tree_block_gb300 as pt

        if s["op"] == "tables":
            lens, counters, row_ptr, slots, positions = pt.cache_tables(s["held"], s["added"], s["tables"], s["ring"], s["counters"], s["page"], s["new"], start=s["start"])
            return dict(lens=lens, counters=counters, row_ptr=row_ptr, slots=slots, positions=positions, tables=s["tables"], ring=s["ring"])
        if s["op"] == "write":
            pt.cache_write(s["K"], s["V"], s["slots"], s["Kc"], s["Vc"])
            return dict(Kc=s["Kc"], Vc=s["Vc"])
        O, LSE = pt.attn_decode(s["Q"], s["Kc"], s["Vc"], s["tables"], s["lens"], s["plan"], workspace=s["workspace"])
        return dict(O=O, LSE=LSE)
    return {"tables": _tables, "write": _write, "decode": _decode}[s["op"]](s)


def _tables(s):
    ps, ring, n = s["page"], s["ring"], s["held"].numel()
    held, added, cap = s["held"].long(), s["added"].long(), ring.numel()
    head, tail = s["counters"][0], s["counters"][1]
    grow = added.clamp(min=0)
    row_ptr = torch.cat([grow.new_zeros(1), grow.cumsum(0)])
    p0, p1 = (held + ps - 1) // ps, (held + added + ps - 1) // ps
    take, back = (p1 - p0).clamp(min=0), (p0 - p1).clamp(min=0)
    col = torch.arange(s["tables"].shape[1], device=held.device)
    at = (head + (take.cumsum(0) - take - p0)[:, None] + col) % cap
    taken = (col >= p0[:, None]) & (col < p1[:, None])
    tables = torch.where(taken, ring[at], s["tables"])
    at = (tail + (back.cumsum(0) - back - p1)[:, None] + col) % cap
    freed = (col >= p1[:, None]) & (col < p0[:, None])
    ring = torch.cat([ring, ring.new_zeros(1)]).scatter(0, torch.where(freed, at, cap).reshape(-1), tables.reshape(-1))[:cap]
    t = torch.arange(s["new"], device=held.device)
    row = torch.searchsorted(row_ptr[1:], t, right=True).clamp(max=n - 1)
    tok = held[row] + t - row_ptr[row]
    real = t < row_ptr[-1]
    page = tables[row, torch.where(real, tok // ps, 0)].long()
    return dict(lens=(held + added).int(), counters=torch.stack([head + take.sum(), tail + back.sum()]), row_ptr=row_ptr.int(),
                slots=torch.where(real, page * ps + tok % ps, -1), positions=torch.where(real, s["start"][row] + tok, 0), tables=tables, ring=ring)


def _write(s):
    slots = s["slots"][:s["real"]]
    page, row = slots // s["page"], slots % s["page"]
    s["Kc"][page, :, row] = s["K"][:s["real"]]
    s["Vc"][page, :, row] = s["V"][:s["real"]]
    return dict(Kc=s["Kc"], Vc=s["Vc"])


def _decode(s):
    lens, q_len, ps, T = s["lens"].long(), s["q_len"], s["page"], s["tokens"]
    Hq, D = s["Q"].shape[1:]
    S, Hkv = s["leaf"].numel(), s["Kc"].shape[1]
    node = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens, output_size=T)
    off = torch.arange(T, device=lens.device) - (lens.cumsum(0) - lens)[node]
    page, row = s["tables"][node, off // ps].long(), off % ps
    K, V = s["Kc"][page, :, row].float(), s["Vc"][page, :, row].float()  # [T, Hkv, D]
    last = lens[s["leaf"]][:, None] - q_len + torch.arange(q_len, device=lens.device)  # each query's place in its leaf
    keep = s["on"][:, node][:, None] & ((node != s["leaf"][:, None])[:, None] | (off <= last[:, :, None]))  # [S, q_len, T]
    Q = s["Q"].float().view(S, q_len, Hkv, Hq // Hkv, D)
    score = torch.einsum("sjhgd,thd->hgsjt", Q, K).mul_(D ** -0.5).masked_fill_(~keep, -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    O = torch.einsum("hgsjt,thd->sjhgd", p, V) / total.permute(2, 3, 0, 1, 4).clamp(min=1e-30)
    return dict(O=O.reshape(S * q_len, Hq, D).to(s["Q"].dtype), LSE=(top + total.log()).reshape(Hq, S * q_len))


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the same by the definition in 64 bits

def work(case):
    ps = case["page"]
    if case["op"] == "tables":
        held, added = _steps(case)
        p0, p1 = -(-held // ps), -(-(held + added) // ps)
        new = int(np.maximum(added, 0).sum()) + case["pad"]
        # lengths, starts, lens, row_ptr; a table and a ring entry for each page that moves; slots and positions
        return dict(bytes=20 * held.size + 8 * int(np.abs(p1 - p0).sum()) + 16 * new + 32, flops=0)
    lens, paths = _tree(case)
    row = case["Hkv"] * case["D"] * (2 if case["type"] == "bf16" else 4)
    if case["op"] == "write":
        n = sum(lens) if case["whole"] else len(paths)
        return dict(bytes=4 * n * row + 8 * (n + case["pad"]), flops=0)
    q = case["q_len"]
    T = sum(lens)
    kept = sum(sum(lens[i] for i in p) * q - q * (q - 1) // 2 for p in paths)
    rows = len(paths) * q
    moved = 2 * T * row + 2 * rows * row * case["Hq"] // case["Hkv"] + 4 * rows * case["Hq"] + 4 * sum(-(-n // ps) + 1 for n in lens)
    return dict(bytes=moved, flops=4 * case["D"] * case["Hq"] * kept)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    ps = case["page"]
    if case["op"] == "write":
        out = {}
        for name in ("K", "V"):
            flat = s[name + "c"].double().transpose(1, 2).flatten(0, 1)  # [slot, head, D]
            flat.index_copy_(0, s["slots"][:s["real"]], s[name].double()[:s["real"]])
            out[name + "c"] = flat.unflatten(0, (-1, ps)).transpose(1, 2).contiguous()
        return out
    Hq, Hkv, D, q = case["Hq"], case["Hkv"], case["D"], case["q_len"]
    lens, paths = _tree(case)
    O = torch.empty(len(paths) * q, Hq, D, dtype=torch.float64, device="cuda")
    LSE = torch.empty(Hq, len(paths) * q, dtype=torch.float64, device="cuda")
    for i, path in enumerate(paths):
        K, V = [], []
        for node in path:
            ids = s["tables"][node, :-(-lens[node] // ps)].long()
            K.append(s["Kc"][ids].transpose(1, 2).flatten(0, 1)[:lens[node]])
            V.append(s["Vc"][ids].transpose(1, 2).flatten(0, 1)[:lens[node]])
        K, V = torch.cat(K).double(), torch.cat(V).double()
        for j in range(q):
            n = K.shape[0] - q + j + 1
            qs = s["Q"][i * q + j].double().view(Hkv, Hq // Hkv, D)
            sc = torch.matmul(qs, K[:n].permute(1, 2, 0)) / D ** 0.5  # [Hkv, group, n]
            LSE[:, i * q + j] = torch.logsumexp(sc, -1).reshape(Hq)
            O[i * q + j] = torch.matmul(torch.softmax(sc, -1), V[:n].transpose(0, 1)).reshape(Hq, D)
    return dict(O=O, LSE=LSE)
