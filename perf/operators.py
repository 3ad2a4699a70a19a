"""The attention operators of a language model's prompt, training and decode steps, as measured cases.

Three operators of the package:
  prefill  fa_fwd_varlen: attention over packed sequences of different lengths, causal, grouped K/V heads
  train    fa_bwd_varlen: its gradients
  decode   fa_fwd_prefix: new tokens of a batch whose sequences share a prefix and have a cache of their own

``run`` computes them in plain torch operations (``own`` false) or with the package's kernels.
"""
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
def _text(lens):
    return ",".join(str(n) for n in lens)


def _lens(text):
    return [int(x) for x in text.split(",")]


def _packed(name, op, H, H_kv, d, q_lens, kv_lens=None, causal=True, fused=False):
    return {"name": name, "op": op, "H": H, "H_kv": H_kv, "d": d, "q_lens": _text(q_lens),
            "kv_lens": _text(q_lens if kv_lens is None else kv_lens), "causal": causal, "fused": fused}


def _decode(name, H, H_kv, d, n_q, prefix, room, lens, causal=False, by_token=False):
    return {"name": name, "op": "decode", "H": H, "H_kv": H_kv, "d": d, "n_q": n_q, "prefix": prefix, "room": room,
            "lens": _text(lens), "causal": causal, "by_token": by_token}


def _spread(seed, n, lo, hi):
    r = random.Random(seed)
    return [int(round(lo * (hi / lo) ** r.random())) for _ in range(n)]


def listed():
    return [
        # One short prompt of an interactive user: latency is all.
        _packed("prefill_short", "prefill", 32, 8, 128, [37]),
        # A server's batch of waiting prompts, one token to 2047, as slices of one projection's output.
        _packed("prefill_batch", "prefill", 32, 8, 128, [1, 2047, 300, 129, 1024, 5, 777, 1500, 64, 411, 1900, 256],
                fused=True),
        # One long prompt: the sizes of this repository's 8k workload, with 8 K/V heads.
        _packed("prefill_8k", "prefill", 32, 8, 128, [8192]),
        # Chunks of prompts whose first part is already in the cache, 64-wide heads.
        _packed("prefill_chunks_d64", "prefill", 16, 4, 64, [512, 100, 17, 333, 256, 1],
                [4000, 1100, 2500, 333, 1000, 3501]),
        # A training batch of documents packed into one row of 8192 tokens.
        _packed("train_packed", "train", 32, 8, 128, [2000, 31, 1024, 1500, 700, 129, 1, 1807, 1000], fused=True),
        # A small model's short documents, every query head with a K/V head of its own.
        _packed("train_short_d64", "train", 16, 16, 64, [100, 255, 1, 420]),
        # Long documents.
        _packed("train_4k", "train", 16, 4, 128, [4096, 4001]),
        # Two users at the start of their answers behind a short system prompt: latency.
        _decode("decode_small", 32, 8, 128, 1, 500, 128, [9, 100]),
        # A batch of answers behind a long shared system prompt.
        _decode("decode_batch64", 32, 8, 128, 1, 8192, 1024, _spread(1, 64, 1, 1024)),
        # Questions on one long document: the length and heads of this repository's 32k decode workload.
        _decode("decode_document", 32, 8, 128, 1, 32768, 2048, _spread(2, 32, 16, 2048)),
        # Four drafted tokens of every sequence checked at once, causal among themselves, cache stored token by token.
        _decode("decode_draft_d64", 16, 4, 64, 4, 1999, 1000, _spread(3, 24, 4, 1000), causal=True, by_token=True),
        # Nothing shared: every sequence has only its own long cache, of its own length.
        _decode("decode_own", 32, 8, 128, 1, 0, 32768, [32768, 20001, 777, 9000, 30000, 1, 15000, 28123]),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["prefill", "train", "decode"])
    d = rng.choice([64, 128, 128])
    H_kv, G = rng.choice([(1, 8), (2, 4), (4, 4), (8, 4), (8, 1), (16, 1), (4, 7), (3, 5), (2, 16)])
    H = H_kv * G
    if op == "decode":
        B = _log(rng, 1, 96)
        n_q = rng.choice([1, 1, 1, 2, 3, 5, 8])
        prefix = rng.choice([0, 1, 1]) * _log(rng, 1, 32768)
        room = _log(rng, max(8, n_q), 4096)
        while B * H * n_q * (prefix + room) > 1 << 25 or B * H_kv * room > 1 << 20:
            prefix, room = prefix // 2, max(8, room // 2)
        lens = [rng.choice([_log(rng, 1, room), rng.randint(0, room)]) for _ in range(B)]
        return _decode("", H, H_kv, d, n_q, prefix, room, lens, n_q > 1 and rng.random() < 0.7, rng.random() < 0.5)
    top = 8192 if op == "prefill" else 4096
    B = _log(rng, 1, 40)
    hi = _log(rng, 4, top)
    kv = [max(1, _log(rng, 1, hi)) for _ in range(B)]
    chunks = rng.random() < 0.35
    q = [rng.choice([n, _log(rng, 1, n)]) if chunks else n for n in kv]
    most = (1 << 30) if op == "prefill" else (1 << 28)
    while B * H * max(q) * max(kv) > most:   # the padded plain form's scores
        if B > 1:
            B -= 1
            q, kv = q[:B], kv[:B]
        else:
            q, kv = [max(1, q[0] // 2)], [max(1, kv[0] // 2)]
    fused = not chunks and rng.random() < 0.5
    return _packed("", op, H, H_kv, d, q, kv, rng.random() < 0.85, fused)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    H, H_kv, d = case["H"], case["H_kv"], case["d"]
    s = {"op": case["op"], "H": H, "H_kv": H_kv, "d": d, "scale": d ** -0.5, "causal": case["causal"]}
    if case["op"] == "decode":
        lens = _lens(case["lens"])
        B, n_q, room, n_p = len(lens), case["n_q"], case["room"], case["prefix"]
        s["q"] = _normal(g, B, H, n_q, d)
        if n_p:
            s["k_prefix"], s["v_prefix"] = _normal(g, H_kv, n_p, d), _normal(g, H_kv, n_p, d)
        else:
            s["k_prefix"] = s["v_prefix"] = None
        if case["by_token"]:   # the cache as [B, room, H_kv, d], seen as [B, H_kv, room, d]
            s["k"], s["v"] = (_normal(g, B, room, H_kv, d).transpose(1, 2) for _ in range(2))
        else:
            s["k"], s["v"] = (_normal(g, B, H_kv, room, d) for _ in range(2))
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        return s
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    Tq, Tk = sum(ql), sum(kl)
    if case["fused"]:          # one projection's output [T, H + 2 H_kv, d]
        qkv = _normal(g, Tq, H + 2 * H_kv, d)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + H_kv], qkv[:, H + H_kv:]
    else:
        s["q"], s["k"], s["v"] = _normal(g, Tq, H, d), _normal(g, Tk, H_kv, d), _normal(g, Tk, H_kv, d)
    s["cu_q"], s["cu_kv"] = _offsets(ql), _offsets(kl)
    s["max_q"], s["max_kv"] = max(ql), max(kl)
    if case["op"] == "train":  # what the forward pass left, and the gradient that arrives
        s["o"], s["lse"] = _prefill(s)
        s["do"] = _normal(g, Tq, H, d)
    return s


# ---------------------------------------------------------------- plain forms
def _pad(x, cu, n):
    """Packed [T, heads, d] as float32 [B, heads, n, d], rows past a sequence's end zero, and which rows exist."""
    at = torch.arange(n, device=x.device)
    live = at < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at).clamp(max=x.shape[0] - 1).long()
    return (x[rows].float() * live[..., None, None]).transpose(1, 2), live


def _unpad(x, cu, total):
    """[B, heads, n, ...] back to packed [total, heads, ...]."""
    t = torch.arange(total, device=x.device)
    b = torch.searchsorted(cu[1:].long().contiguous(), t, right=True)
    return x.transpose(1, 2)[b, t - cu[b]]


def _visible(s):
    """[B, 1, 1, max_q, max_kv]: which key a row sees."""
    n_q, n_kv = (s[c][1:] - s[c][:-1] for c in ("cu_q", "cu_kv"))
    i = torch.arange(s["max_q"], device=DEV)[:, None]
    j = torch.arange(s["max_kv"], device=DEV)
    see = (i < n_q[:, None, None]) & (j < n_kv[:, None, None])
    if s["causal"]:
        see = see & (j <= i + (n_kv - n_q)[:, None, None])
    return see[:, None, None]


def _heads(x, H_kv):
    """[B, H, n, d] -> [B, H_kv, G, n, d]."""
    return x.reshape(x.shape[0], H_kv, -1, *x.shape[2:])


def _softmax(x):
    """Rows' weights and log-sum-exp; a row of -inf alone gets weights 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l == 0, torch.ones_like(l), l), (m + l.log()).squeeze(-1)


def _prefill(s):
    q, _ = _pad(s["q"], s["cu_q"], s["max_q"])
    k, _ = _pad(s["k"], s["cu_kv"], s["max_kv"])
    v, _ = _pad(s["v"], s["cu_kv"], s["max_kv"])
    x = _heads(q, s["H_kv"]) @ k[:, :, None].transpose(-1, -2)
    x = (x * s["scale"]).masked_fill_(~_visible(s), float("-inf"))
    p, lse = _softmax(x)
    del x
    o = (p @ v[:, :, None]).flatten(1, 2)
    T = s["q"].shape[0]
    return (_unpad(o, s["cu_q"], T).to(torch.bfloat16),
            _unpad(lse.flatten(1, 2), s["cu_q"], T).t().contiguous())


def _train(s):
    Hk = s["H_kv"]
    q, do, o = (_heads(_pad(s[n], s["cu_q"], s["max_q"])[0], Hk) for n in ("q", "do", "o"))
    k, v = (_pad(s[n], s["cu_kv"], s["max_kv"])[0][:, :, None] for n in ("k", "v"))
    lse = _heads(_pad(s["lse"].t()[..., None], s["cu_q"], s["max_q"])[0], Hk)
    p = ((q @ k.transpose(-1, -2)) * s["scale"] - lse).exp_()
    p.masked_fill_(~_visible(s), 0.0)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = ((ds @ k) * s["scale"]).flatten(1, 2)
    dk = (ds.transpose(-1, -2) @ q).sum(2) * s["scale"]
    return tuple(_unpad(x, s[c], s[n].shape[0]).to(torch.bfloat16)
                 for x, c, n in ((dq, "cu_q", "q"), (dk, "cu_kv", "k"), (dv, "cu_kv", "v")))


def _decode_plain(s):
    B, H, n_q, d = s["q"].shape
    Hk = s["H_kv"]
    G = H // Hk
    q = s["q"].float().reshape(B, Hk, G * n_q, d)
    k, v = s["k"].float(), s["v"].float()
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).reshape(B, Hk, G, n_q, -1)
    j = torch.arange(k.shape[2], device=DEV)
    end = s["lens"][:, None].expand(B, n_q)
    if s["causal"]:
        end = end - (n_q - 1) + torch.arange(n_q, device=DEV)
    live = (j < end[..., None])[:, None, None]
    x.masked_fill_(~live, float("-inf"))
    v = torch.where((j < s["lens"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    if s["k_prefix"] is not None:
        kp, vp = s["k_prefix"].float(), s["v_prefix"].float()
        rows = q.transpose(0, 1).reshape(Hk, B * G * n_q, d)
        xp = (rows @ kp.transpose(-1, -2)).mul_(s["scale"]).reshape(Hk, B, G, n_q, -1).transpose(0, 1)
        p, lse = _softmax(torch.cat([xp, x], -1))
        n_p = kp.shape[1]
        pp = p[..., :n_p].transpose(0, 1).reshape(Hk, B * G * n_q, n_p)
        o = (pp @ vp).reshape(Hk, B, G * n_q, d).transpose(0, 1) + p[..., n_p:].reshape(B, Hk, G * n_q, -1) @ v
    else:
        p, lse = _softmax(x)
        o = p.reshape(B, Hk, G * n_q, -1) @ v
    return o.reshape(B, H, n_q, d).to(torch.bfloat16), lse.reshape(B, H, n_q)


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        from exact_io_aware_34_gb300 import fa
        if s["op"] == "prefill":
            return fa.fa_fwd_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_kv"], scale=s["scale"],
                                    causal=s["causal"])
        if s["op"] == "train":
            return fa.fa_bwd_varlen(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["cu_q"], s["cu_kv"],
                                    scale=s["scale"], causal=s["causal"])
        return fa.fa_fwd_prefix(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["lens"], scale=s["scale"],
                                causal=s["causal"])
    return {"prefill": _prefill, "train": _train, "decode": _decode_plain}[s["op"]](s)


# ---------------------------------------------------------------- what a pass cannot do without
def _seen(n_q, n_kv, causal):
    """(row, key) pairs of one sequence."""
    if not causal:
        return n_q * n_kv
    return sum(max(0, min(n_kv, i + 1 + n_kv - n_q)) for i in range(n_q))


def work(case):
    H, H_kv, d = case["H"], case["H_kv"], case["d"]
    if case["op"] == "decode":
        lens, n_q, n_p = _lens(case["lens"]), case["n_q"], case["prefix"]
        rows = len(lens) * n_q * H
        pairs = len(lens) * n_q * n_p + sum(_seen(n_q, n, case["causal"]) for n in lens)
        keys = H_kv * (n_p + sum(lens))
        return {"bytes": 2 * 2 * rows * d + 4 * rows + 2 * 2 * keys * d + 4 * len(lens), "flops": 4 * d * H * pairs}
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    rows, keys = sum(ql) * H, sum(kl) * H_kv
    pairs = H * sum(_seen(a, b, case["causal"]) for a, b in zip(ql, kl))
    if case["op"] == "prefill":
        return {"bytes": 2 * 2 * rows * d + 2 * 2 * keys * d + 4 * rows, "flops": 4 * d * pairs}
    return {"bytes": 2 * 4 * rows * d + 2 * 4 * keys * d + 4 * rows, "flops": 10 * d * pairs}


# ---------------------------------------------------------------- in 64 bits
def _one_head(q, k, v, scale, shift):
    """One head's attention in float64; row i sees keys j <= i + shift (None: all)."""
    x = (q @ k.T) * scale
    if shift is not None:
        x[torch.ones_like(x, dtype=torch.bool).triu(shift + 1)] = float("-inf")
    lse = torch.logsumexp(x, -1) if x.shape[1] else torch.full((x.shape[0],), float("-inf"), dtype=x.dtype, device=DEV)
    w = torch.where(lse[:, None].isinf(), torch.zeros_like(x), (x - lse[:, None]).exp())
    return w @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    H, H_kv, G, scale = s["H"], s["H_kv"], s["H"] // s["H_kv"], s["scale"]
    f = torch.float64
    if case["op"] == "decode":
        lens, n_q = _lens(case["lens"]), case["n_q"]
        o = torch.zeros(s["q"].shape, dtype=f, device=DEV)
        lse = torch.zeros(s["q"].shape[:-1], dtype=f, device=DEV)
        for h in range(H_kv):
            n_p = case["prefix"]
            kp = s["k_prefix"][h].to(f) if n_p else s["q"].new_zeros((0, s["d"]), dtype=f)
            vp = s["v_prefix"][h].to(f) if n_p else kp
            for b, n in enumerate(lens):
                k, v = (torch.cat([a, s[c][b, h, :n].to(f)]) for a, c in ((kp, "k"), (vp, "v")))
                for i in range(n_q):
                    end = n_p + (max(0, n - (n_q - 1 - i)) if case["causal"] else n)
                    hs = slice(h * G, h * G + G)
                    o[b, hs, i], lse[b, hs, i] = _one_head(s["q"][b, hs, i].to(f), k[:end], v[:end], scale, None)
        return o, lse
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    out = [torch.zeros(s[n].shape, dtype=f, device=DEV) for n in ("q", "k", "v")]
    lse = torch.zeros((H, s["q"].shape[0]), dtype=f, device=DEV)
    a = c = 0
    for n, m in zip(ql, kl):
        r, t = slice(a, a + n), slice(c, c + m)
        for h in range(H):
            q, k, v = s["q"][r, h].to(f), s["k"][t, h // G].to(f), s["v"][t, h // G].to(f)
            shift = m - n if case["causal"] else None
            if case["op"] == "prefill":
                out[0][r, h], lse[h, r] = _one_head(q, k, v, scale, shift)
                continue
            p = ((q @ k.T) * scale - s["lse"][h, r, None].to(f)).exp()
            if shift is not None:
                p = p.tril(shift)
            do = s["do"][r, h].to(f)
            ds = p * (do @ v.T - (do * s["o"][r, h].to(f)).sum(-1, keepdim=True))
            out[0][r, h] = scale * (ds @ k)
            out[1][t, h // G] += scale * (ds.T @ q)
            out[2][t, h // G] += p.T @ do
        a, c = a + n, c + m
    return (out[0], lse) if case["op"] == "prefill" else tuple(out)
