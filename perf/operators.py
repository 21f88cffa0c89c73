"""Serving operators around a compressed K/V cache, as cases that can be timed and compared.

Four operators: causal attention over packed prompts (before anything is compressed), writing keys and values
into a paged 8-bit cache, reading rows of that cache back, and attention of a few drafted tokens per sequence
(a tree; one token is the ordinary decode step) over that cache.  ``run`` computes them with elementary torch
operations where ``own`` is false, and through this repository's package where it is true.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    p = {"op": "prompt", "spread": True}
    t = {"op": "tree", "spread": True}
    return [
        # a few short requests that arrive together: latency counts
        dict(p, name="prompt-short", nseq=6, total=331, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a mixed batch of prompts of very different lengths
        dict(p, name="prompt-mixed", nseq=16, total=16411, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # one long document
        dict(p, name="prompt-long", nseq=1, total=32768, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a smaller model: a key head for every query head, 64 channels, fp16
        dict(p, name="prompt-d64", nseq=9, total=8191, Hq=16, Hkv=16, d=64, dtype="f16"),
        # one user, one token, a short chat: the smallest decode step
        dict(t, name="tree-one-token", B=1, n=1, ctx=1000, page=16, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # the decode step of the long-context configuration (batch 8, 131072 tokens each)
        dict(t, name="tree-decode-long", B=8, n=1, ctx=131071, page=64, Hq=32, Hkv=8, d=128, dtype="bf16", spread=False),
        # verification of a drafted tree of 16 tokens, ragged batch
        dict(t, name="tree-draft-16", B=16, n=16, ctx=16000, page=16, Hq=32, Hkv=8, d=128, dtype="bf16"),
        # a wide tree of 61 tokens for a few users with 64-channel heads, fp16
        dict(t, name="tree-draft-61", B=4, n=61, ctx=30001, page=64, Hq=16, Hkv=4, d=64, dtype="f16"),
        # the keys and values of one decode step of 64 users
        dict(op="write", name="write-step", n=64, Hkv=8, d=128, dtype="bf16"),
        # the keys and values of a long prompt
        dict(op="write", name="write-prompt", n=65537, Hkv=8, d=128, dtype="bf16"),
        # the rows of a few pages, on their way into the 4-bit cache
        dict(op="read", name="read-pages", n=1024, d=128, dtype="bf16"),
        # a whole context of 131072 tokens and 8 heads
        dict(op="read", name="read-context", n=1048576, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "tree", "write", "read"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hq, Hkv = rng.choice([(32, 8), (16, 16), (8, 1), (12, 4), (28, 4), (5, 5), (16, 2)])
    d = rng.choice([64, 128, 128, 80, 96])
    if op == "prompt":
        total = _log(rng, 40, 16000)
        return dict(op=op, nseq=min(total, _log(rng, 1, 40)), total=total, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, spread=rng.random() < 0.7)
    if op == "tree":
        B = _log(rng, 1, 48)
        return dict(op=op, B=B, n=rng.choice([1, 1, 2, 5, 8, 13, 16, 24, 32, 48, 64]), ctx=_log(rng, 20, min(100000, 400000 // B)),
                    page=rng.choice([8, 16, 32, 64, 256]), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, spread=rng.random() < 0.7)
    if op == "write":
        return dict(op=op, n=_log(rng, 1, 60000), Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "f16", "f32"]))
    return dict(op=op, n=_log(rng, 1, 1000000), d=d, dtype=rng.choice(["bf16", "f16", "f32"]))


def _lengths(case):
    """The sequences' lengths: a property of the case (its work depends on them), not of the seed."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    if case["op"] == "prompt":
        n, total = case["nseq"], case["total"]
        w = [math.exp(r.gauss(0.0, 1.0)) if case["spread"] else 1.0 for _ in range(n)]
        cut = [0] + [int(round(total * sum(w[: i + 1]) / sum(w))) for i in range(n)]
        return [cut[i + 1] - cut[i] for i in range(n)]
    ctx = [max(0, int(case["ctx"] * r.random())) if case["spread"] and b else case["ctx"] for b in range(case["B"])]
    drafts = [r.randint(1, case["n"]) if case["spread"] and b else case["n"] for b in range(case["B"])]
    return ctx, drafts


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    d = case["d"]
    if case["op"] == "prompt":
        T, Hq, Hkv = case["total"], case["Hq"], case["Hkv"]
        pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
        return {"bytes": T * (2 * Hq + 2 * Hkv) * d * e + T * Hq * 4, "flops": 4 * d * Hq * pairs}
    if case["op"] == "tree":
        ctx, drafts = _lengths(case)
        Hq, Hkv = case["Hq"], case["Hkv"]
        rows = sum(drafts) * Hq
        keys = sum(c + m for c, m in zip(ctx, drafts)) * Hkv
        pairs = sum(m * c + m * (m + 1) // 2 for c, m in zip(ctx, drafts)) * Hq
        return {"bytes": keys * 2 * (d + 4) + rows * (2 * d * e + 4), "flops": 4 * d * pairs}
    if case["op"] == "write":
        N = case["n"] * case["Hkv"]
        return {"bytes": N * (2 * (d * e + d + 4) + 8), "flops": 0}
    N = case["n"]
    return {"bytes": N * (2 * (d * e + d + 4) + 8), "flops": 0}


# ------------------------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _codes(g, rows, d):
    """Codes of roughly normal values, the largest of a row near 127."""
    return _randn(g, rows, d, dtype=torch.float16).mul_(40).round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, rows):
    """Scales of rows whose values have sizes around one, not all alike."""
    return _randn(g, rows).mul_(0.4).exp_().mul_(1.0 / 40)


def prepare(case, seed):
    g = _gen(seed)
    d, ty = case["d"], TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "prompt":
        T, Hq, Hkv = case["total"], case["Hq"], case["Hkv"]
        cu = [0]
        for n in _lengths(case):
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["q"] = (2 * _randn(g, T, Hq, d)).to(ty)
        # keys and values with channels of different sizes
        s["k"] = (_randn(g, T, Hkv, d) * (0.5 * _randn(g, Hkv, d)).exp()).to(ty)
        s["v"] = (_randn(g, T, Hkv, d) * (0.5 * _randn(g, Hkv, d)).exp()).to(ty)
        s["out"] = torch.zeros(T, Hq, d, dtype=ty, device=DEV)
        s["lse"] = torch.zeros(T, Hq, dtype=torch.float32, device=DEV)
    elif case["op"] == "tree":
        B, n, Hq, Hkv, page = case["B"], case["n"], case["Hq"], case["Hkv"], case["page"]
        ctx, drafts = _lengths(case)
        pages = -(-(max(c + m for c, m in zip(ctx, drafts))) // page)
        pool = B * Hkv * pages + 3
        s["table"] = torch.randperm(pool, generator=g, device=DEV)[: B * Hkv * pages].reshape(B * Hkv, pages).to(torch.int32)
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
        s["drafts"] = torch.tensor(drafts, dtype=torch.int32, device=DEV)
        # every drafted token has an earlier one as its parent, or hangs on the context; it sees its ancestors and itself
        parent = torch.stack([torch.randint(-1, max(i, 1), (B,), generator=g, device=DEV) if i else torch.full((B,), -1, device=DEV) for i in range(n)], 1)
        sees = torch.eye(n, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
        for i in range(1, n):
            up = sees[torch.arange(B, device=DEV), parent[:, i].clamp(min=0)] & (parent[:, i] >= 0)[:, None]
            sees[:, i] |= up
        words = -(-n // 32)
        bits = torch.zeros(B, n, words * 32, dtype=torch.int64, device=DEV)
        bits[:, :, :n] = sees
        packed = (bits.reshape(B, n, words, 32) << torch.arange(32, device=DEV)).sum(-1)
        s["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
        s["q"] = (2 * _randn(g, B, n, Hq, d)).to(ty)
        s["kcodes"], s["kscales"] = _codes(g, pool * page, d), _scales(g, pool * page)
        s["vcodes"], s["vscales"] = _codes(g, pool * page, d), _scales(g, pool * page)
        s["out"] = torch.zeros(B, n, Hq, d, dtype=ty, device=DEV)
        s["lse"] = torch.zeros(B, n, Hq, dtype=torch.float32, device=DEV)
    else:
        rows = case["n"] * case.get("Hkv", 1)
        pool = rows + 64
        slots = torch.randperm(pool, generator=g, device=DEV)[:rows]
        if case["op"] == "write":
            s["slots"] = slots.reshape(case["n"], case["Hkv"])
            for x in "kv":
                s[x] = (_randn(g, case["n"], case["Hkv"], d) * (0.5 * _randn(g, case["Hkv"], d)).exp()).to(ty)
                s[x + "codes"] = torch.zeros(pool, d, dtype=torch.int8, device=DEV)
                s[x + "scales"] = torch.zeros(pool, dtype=torch.float32, device=DEV)
        else:
            s["slots"] = slots
            for x in "kv":
                s[x + "codes"], s[x + "scales"] = _codes(g, pool, d), _scales(g, pool)
                s[x + "out"] = torch.zeros(rows, d, dtype=ty, device=DEV)
    if own:
        import compressed_kv_cache_turboquant_b200 as tq
        s["h"] = tq.tq_create_kv8(d)
        need = 0
        if case["op"] == "prompt":
            need = tq.tq_attn_prompt_workspace(s["h"], case["nseq"], case["total"], case["Hq"], case["Hkv"])
        elif case["op"] == "tree":
            need = tq.tq_attn_tree_workspace(s["h"], case["B"], case["n"], case["Hq"], case["Hkv"])
        s["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------ one pass

def _attend(S, sees, V):
    """Rows of logits S against values V where `sees`; a row that sees nothing gives zeros and a log-sum of -inf."""
    S = S.masked_fill_(~sees, -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = S.sub_(m).exp_()
    l = P.sum(-1, keepdim=True)
    out = torch.matmul(P, V) / torch.where(l == 0, torch.ones_like(l), l)
    return out, (m + l.log()).squeeze(-1)


def _plain_prompt(s):
    T, Hkv, d = s["total"], s["Hkv"], s["d"]
    G = s["Hq"] // Hkv
    at = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu"].long(), at, right=True)
    sees = (seq[:, None] == seq[None, :]) & (at[:, None] >= at[None, :])
    out, lse = torch.zeros_like(s["out"]), torch.zeros_like(s["lse"])
    for h in range(Hkv):  # one key head at a time: the logits of all of them together may not fit
        q = s["q"][:, h * G:(h + 1) * G].float().transpose(0, 1)
        o, e = _attend(torch.matmul(q, s["k"][:, h].float().T).mul_(1 / math.sqrt(d)), sees, s["v"][:, h].float())
        out[:, h * G:(h + 1) * G] = o.transpose(0, 1).to(out.dtype)
        lse[:, h * G:(h + 1) * G] = e.T
    return {"out": out, "lse": lse}


def _plain_tree(s):
    B, n, Hq, Hkv, d, page = (s[k] for k in ("B", "n", "Hq", "Hkv", "d", "page"))
    G = Hq // Hkv
    ctx, drafts = s["ctx"].long(), s["drafts"].long()
    t = torch.arange(s["table"].shape[1] * page, device=DEV)
    rows = s["table"].long()[:, t // page] * page + t % page
    K = s["kcodes"][rows].float().mul_(s["kscales"][rows][..., None])
    V = s["vcodes"][rows].float().mul_(s["vscales"][rows][..., None])
    j = t[None, :] - ctx[:, None]  # place among the drafted tokens
    at = j.clamp(0, n - 1)[:, None, :].expand(B, n, -1)
    bit = (s["mask"].long().gather(2, at // 32) >> (at % 32)) & 1
    sees = (j < 0)[:, None, :] | ((bit == 1) & ((j >= 0) & (j < drafts[:, None]))[:, None, :])
    sees = sees[:, None, :, None, :].expand(B, Hkv, n, G, len(t)).reshape(B * Hkv, n * G, len(t))
    q = s["q"].float().reshape(B, n, Hkv, G, d).transpose(1, 2).reshape(B * Hkv, n * G, d)
    out, lse = _attend(torch.matmul(q, K.transpose(1, 2)).mul_(1 / math.sqrt(d)), sees, V)
    out = out.reshape(B, Hkv, n, G, d).transpose(1, 2).reshape(B, n, Hq, d)
    lse = lse.reshape(B, Hkv, n, G).transpose(1, 2).reshape(B, n, Hq)
    live = torch.arange(n, device=DEV)[None, :] < drafts[:, None]
    out = torch.where(live[..., None, None], out, torch.zeros_like(out))
    return {"out": out.to(s["out"].dtype), "lse": torch.where(live[..., None], lse, torch.zeros_like(lse))}


def _plain_write(s):
    got = {}
    rows = s["slots"].reshape(-1)
    for x in "kv":
        a = s[x].reshape(-1, s["d"]).double()  # in 64 bits: a quotient next to a border between two codes falls on its own side
        scale = (a.abs().amax(1) / 127).float()
        code = torch.where(scale[:, None] > 0, a / scale.double()[:, None], torch.zeros_like(a)).round().clamp(-127, 127)
        s[x + "codes"][rows] = code.to(torch.int8)
        s[x + "scales"][rows] = scale
        got[x + "codes"], got[x + "scales"] = s[x + "codes"], s[x + "scales"]
    return got


def _plain_read(s):
    return {x: (s[x + "codes"][s["slots"]].float() * s[x + "scales"][s["slots"]][:, None]).to(s[x + "out"].dtype) for x in "kv"}


def run(s):
    if not own:
        return {"prompt": _plain_prompt, "tree": _plain_tree, "write": _plain_write, "read": _plain_read}[s["op"]](s)
    import compressed_kv_cache_turboquant_b200 as tq
    if s["op"] == "prompt":
        tq.tq_attn_prompt(s["h"], s["q"], s["k"], s["v"], s["cu"], 1 / math.sqrt(s["d"]), s["out"], lse=s["lse"], workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    cache = [s[k] for k in ("kcodes", "kscales", "vcodes", "vscales")]
    if s["op"] == "tree":
        tq.tq_attn_tree(s["h"], s["q"], s["Hkv"], s["ctx"], s["table"], s["page"], *cache, 1 / math.sqrt(s["d"]), s["out"],
                        lse=s["lse"], mask=s["mask"], draft_lens=s["drafts"], workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "write":
        tq.tq_quant_kv8(s["h"], s["k"], s["v"], s["slots"], *cache)
        return dict(zip(("kcodes", "kscales", "vcodes", "vscales"), cache))
    tq.tq_dequant_kv8(s["h"], s["slots"], *cache, s["kout"], s["vout"])
    return {"k": s["kout"], "v": s["vout"]}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_rows(q, K, V, sees):
    """softmax(q K^T) V and its log-sum in 64 bits for one head: q [rows][d] with the scale in it."""
    z = q @ K.T
    z[~sees] = -math.inf
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - lse[:, None])
    w[~sees] = 0
    return w @ V, lse


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "read":
        return {x: s[x + "scales"][s["slots"]].double()[:, None] * s[x + "codes"][s["slots"]].double() for x in "kv"}
    if case["op"] == "write":
        got = {}
        for x in "kv":
            scale = s[x + "scales"].double()
            scale[s["slots"]] = s[x].double().abs().max(-1).values / 127
            got[x + "codes"], got[x + "scales"] = None, scale
        return got
    Hq, Hkv = case["Hq"], case["Hkv"]
    G = Hq // Hkv
    out, lse = s["out"].double(), s["lse"].double()
    if case["op"] == "prompt":
        if sum(n * n for n in _lengths(case)) * Hq * d > 6e12:
            return None
        end = 0
        for n in _lengths(case):
            a, end = end, end + n
            for h in range(Hq):
                K, V = s["k"][a:end, h // G].double(), s["v"][a:end, h // G].double()
                for i in range(0, n, 4096):
                    m = min(n, i + 4096)
                    sees = torch.ones(m - i, m, dtype=torch.bool, device=DEV).tril(i)
                    o, e = _exact_rows(s["q"][a + i:a + m, h].double() / math.sqrt(d), K[:m], V[:m], sees)
                    out[a + i:a + m, h], lse[a + i:a + m, h] = o, e
        return {"out": out, "lse": lse}
    ctx, drafts = _lengths(case)
    for b in range(case["B"]):
        T, m = ctx[b] + drafts[b], drafts[b]
        sees = torch.ones(m, T, dtype=torch.bool, device=DEV)
        for i in range(m):
            words = [int(w) & 0xFFFFFFFF for w in s["mask"][b, i].tolist()]
            sees[i, ctx[b]:] = torch.tensor([bool(words[j // 32] >> (j % 32) & 1) for j in range(m)], device=DEV)
        for h in range(Hkv):
            pages = s["table"][b * Hkv + h].long()
            rows = (pages[:, None] * case["page"] + torch.arange(case["page"], device=DEV)).reshape(-1)[:T]
            K = s["kcodes"][rows].double() * s["kscales"][rows].double()[:, None]
            V = s["vcodes"][rows].double() * s["vscales"][rows].double()[:, None]
            for u in range(h * G, h * G + G):
                o, e = _exact_rows(s["q"][b, :m, u].double() / math.sqrt(d), K, V, sees)
                out[b, :m, u], lse[b, :m, u] = o, e
    return {"out": out, "lse": lse}
