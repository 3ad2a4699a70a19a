"""The operators of a language model that answers from a paged 8-bit cache, as measured cases.

Three operators of the package:
  rope    fa_rope: rotary positions on queries and keys, and the gradient of that
  append  fa_kv_append: new keys (rotated on the way) and values into pages held in 8 bits, queries rotated beside them
  paged   fa_fwd_paged: attention of new tokens over such pages, with a scale for each page and head
and ``step``, the last two one after the other as a decode step makes them.

``run`` computes them in plain torch operations (``own`` false) or with the package's kernels.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = 448.0          # largest e4m3 value
LEAST = -100         # a page's scale is 2^e with e at least this


# ---------------------------------------------------------------- cases
def _text(lens):
    return ",".join(str(n) for n in lens)


def _lens(text):
    return [int(x) for x in text.split(",")]


def _rope(name, T, heads, heads_y, d, rot, first, doc, interleaved=False, transpose=False, fused=False, base=1e4, factor=1.0):
    return {"name": name, "op": "rope", "T": T, "heads": heads, "heads_y": heads_y, "d": d, "rot": rot, "first": first,
            "doc": doc, "interleaved": interleaved, "transpose": transpose, "fused": fused, "base": base, "factor": factor}


def _cache(name, op, H, H_kv, d, page, new, lens, causal=True, by_token=False, rot=0, interleaved=False, base=1e4):
    return {"name": name, "op": op, "H": H, "H_kv": H_kv, "d": d, "page": page, "new": _text(new), "lens": _text(lens),
            "causal": causal, "by_token": by_token, "rot": rot, "interleaved": interleaved, "base": base}


def _spread(seed, n, lo, hi):
    r = random.Random(seed)
    return [int(round(lo * (hi / lo) ** r.random())) for _ in range(n)]


def listed():
    prompts = [1, 2047, 300, 129, 1024, 5, 777, 1500, 64, 411, 1900, 256]
    batch = _spread(1, 64, 1, 8192)
    return [
        # A short prompt of one user at the far end of a long conversation: latency is all.
        _rope("rope_short", 37, 32, 8, 128, 128, 1000003, 37, base=5e5),
        # A training batch of documents packed into 8192 rows: queries and keys inside one projection's output.
        _rope("rope_train", 8192, 40, 0, 128, 128, 0, 1807, fused=True),
        # The gradient for a small model that rotates half of each head, neighbours in pairs, scaled for a longer context.
        _rope("rope_grad_partial", 16001, 16, 4, 64, 32, 0, 4001, interleaved=True, transpose=True, factor=1.1386),
        # The next token of two users: latency.
        _cache("append_small", "append", 32, 8, 128, 64, [1, 1], [510, 101], rot=128),
        # The next token of every sequence of a batch, each into its own last page.
        _cache("append_batch64", "append", 32, 8, 128, 64, [1] * 64, batch, rot=128),
        # A server's batch of prompts written into a fresh cache, short pages.
        _cache("append_prompts", "append", 32, 8, 128, 16, prompts, prompts, rot=128),
        # Two users at the start of their answers: latency.
        _cache("paged_small", "paged", 32, 8, 128, 64, [1, 1], [509, 600]),
        # A batch of answers of very different lengths.
        _cache("paged_batch64", "paged", 32, 8, 128, 64, [1] * 64, batch),
        # Long caches: the lengths and heads of this repository's 32k decode workload.
        _cache("paged_long", "paged", 32, 8, 128, 128, [1] * 8, [32768, 20001, 777, 9000, 30000, 1, 15000, 28123]),
        # Four drafted tokens of every sequence checked at once, 64-wide heads, short pages stored token by token.
        _cache("paged_draft_d64", "paged", 16, 4, 64, 16, [4] * 24, _spread(3, 24, 4, 4000), by_token=True),
        # Chunks of prompts whose first part is already in the cache, and single tokens beside them.
        _cache("paged_chunks", "paged", 32, 8, 128, 64, [1024, 1, 300, 1, 17, 1], [8192, 3501, 2500, 1000, 333, 64]),
        # One whole attention step of a batch: append, rotate, attend.
        _cache("step_batch32", "step", 32, 8, 128, 32, [1] * 32, _spread(4, 32, 16, 16384), rot=64, interleaved=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "paged", "paged", "paged", "step"])
    H_kv, G = rng.choice([(1, 8), (2, 4), (4, 4), (8, 4), (8, 1), (16, 1), (4, 7), (3, 5), (2, 16)])
    base = rng.choice([1e4, 1e4, 5e5])
    if op == "rope":
        d = rng.choice([64, 128, 128, 96, 256])
        heads, heads_y = H_kv * G, rng.choice([0, H_kv])
        T = _log(rng, 1, min(16384, 8192 * 40 * 128 // ((heads + heads_y) * d)))
        rot = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
        return _rope("", T, heads, heads_y, d, rot, rng.choice([0, _log(rng, 1, 1 << 20)]), _log(rng, 1, T),
                     rng.random() < 0.5, rng.random() < 0.4, heads_y == 0 and rng.random() < 0.5, base,
                     rng.choice([1.0, 1.0, 1.25]))
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    B = _log(rng, 1, 96)
    top = _log(rng, 2, 32768)
    chunks = op != "step" and rng.random() < 0.4
    lens = [rng.choice([_log(rng, 1, top), rng.randint(1, top)]) for _ in range(B)]
    if chunks:
        new = [rng.choice([1, _log(rng, 1, min(n, 2048))]) for n in lens]
    else:
        k = rng.choice([1, 1, 1, 2, 3, 5, 8])
        new = [min(k, n) for n in lens]
    H = H_kv * G
    # No more than the largest listed cases read, write or (as a padded plain form) multiply.
    while (B * H * max(new) * max(lens) > 1 << 28 or B * max(lens) * H_kv * d > 1 << 27
           or sum(new) * (H + 2 * H_kv) * d > 8000 * 48 * 128):
        if B > 1:
            B //= 2
            lens, new = lens[:B], new[:B]
        else:
            lens = [max(1, lens[0] // 2)]
            new = [min(max(1, new[0] // 2), lens[0])]
    rot = 0 if op == "paged" else rng.choice([d, d, d // 2, 0 if op == "append" else d])
    return _cache("", op, H, H_kv, d, page, new, lens, rng.random() < 0.85 or op == "step", rng.random() < 0.4, rot,
                  rng.random() < 0.5, base)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _frequencies(rot, base):
    """Radians per position of each of the rot / 2 pairs."""
    return base ** (torch.arange(rot // 2, device=DEV, dtype=torch.float64) * (-2.0 / rot))


def _least_scale(amax):
    """The smallest power of two, 2^LEAST at least, by which values up to amax fit e4m3."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > TOP / 512).to(e.dtype)
    e = torch.where(amax > 0, e.clamp(min=LEAST), torch.full_like(e, LEAST))
    return torch.ldexp(torch.ones_like(amax), e)


def _filled(g, n_pages, H_kv, page, d, by_token):
    """A cache whose pages are full: codes [n_pages, H_kv, page, d] and scales [n_pages, H_kv]."""
    x = torch.randn((n_pages, H_kv, page, d), generator=g, device=DEV, dtype=torch.float32)
    x.mul_(torch.randn((n_pages, H_kv, 1, 1), generator=g, device=DEV).mul_(0.4).exp_())   # blocks of unequal size
    scale = _least_scale(x.abs().amax((2, 3)))
    x.div_(scale[:, :, None, None])
    if by_token:   # stored as [n_pages, page, H_kv, d]
        return x.transpose(1, 2).contiguous().to(E4M3).transpose(1, 2), scale
    return x.to(E4M3), scale


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "rope":
        T, heads, heads_y, d = case["T"], case["heads"], case["heads_y"], case["d"]
        if case["fused"]:      # the first heads of a projection's output [T, heads + heads // 4, d]
            s["x"], s["y"] = _normal(g, T, heads + max(1, heads // 4), d)[:, :heads], None
        else:
            s["x"], s["y"] = _normal(g, T, heads, d), _normal(g, T, heads_y, d) if heads_y else None
        s["positions"] = (torch.arange(T, device=DEV) % case["doc"] + case["first"]).to(torch.int32)
        s["inv_freq"] = _frequencies(case["rot"], case["base"])
        return s
    H, H_kv, d, page = case["H"], case["H_kv"], case["d"], case["page"]
    new, lens = _lens(case["new"]), _lens(case["lens"])
    B, T = len(new), sum(new)
    s["scale"], s["max_q"], s["max_kv"] = d ** -0.5, max(new), max(lens)
    s["q"] = _normal(g, T, H, d)
    if case["op"] != "paged":
        kv = _normal(g, T, 2 * H_kv, d)      # the key and value parts of one projection's output
        s["k"], s["v"] = kv[:, :H_kv], kv[:, H_kv:]
    used = [-(-n // page) for n in lens]
    n_pages = sum(used) + 3                  # pages of no sequence stay as they are
    s["k_cache"], s["k_scale"] = _filled(g, n_pages, H_kv, page, d, case["by_token"])
    s["v_cache"], s["v_scale"] = _filled(g, n_pages, H_kv, page, d, case["by_token"])
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(max(used), device=DEV)
    used = torch.tensor(used, device=DEV)
    first = used.cumsum(0) - used
    s["page_table"] = torch.where(at < used[:, None], order[(first[:, None] + at).clamp(max=n_pages - 1)],
                                  torch.full((), -1, dtype=torch.int32, device=DEV)).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s["inv_freq"] = _frequencies(case["rot"], case["base"]) if case["rot"] else None
    return s


# ---------------------------------------------------------------- plain forms
def _turned(x, positions, inv_freq, interleaved, transpose=False, factor=1.0):
    """x [T, heads, d] in float32 with its first 2 * len(inv_freq) columns rotated; angles in 64 bits."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq
    c, s = ((f * factor).float()[:, None] for f in (angle.cos(), angle.sin()))
    if transpose:
        s = -s
    x = x.float()
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    u, w = a * c - b * s, a * s + b * c
    r = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([r, x[..., 2 * half:]], -1)


def _rope_plain(s):
    out = [_turned(x, s["positions"], s["inv_freq"], s["interleaved"], s["transpose"], s["factor"]).to(torch.bfloat16)
           for x in (s["x"], s["y"]) if x is not None]
    return tuple(out)


def _places(s):
    """Sequence, position in it and page of every new token."""
    t = torch.arange(s["q"].shape[0], device=DEV)
    cu, lens = s["cu"].long(), s["lens"].long()
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = t - cu[b + 1] + lens[b]
    return b, pos, s["page_table"][b, pos // s["page"]].long()


def _store(x, cache, scale, s, b, pos, pid):
    """x [T, H_kv, d] in float32 into its pages; a page's old rows are brought to its new scale."""
    page = s["page"]
    n_new = (s["cu"][1:] - s["cu"][:-1]).long()
    before = s["lens"].long() - n_new                       # rows that were there
    kept = before % page * (n_new > 0)                      # old rows of the first page written, by sequence
    need = torch.zeros_like(scale)
    need.scatter_reduce_(0, pid[:, None].expand(-1, scale.shape[1]), x.abs().amax(-1), "amax")
    # The page of each sequence that may hold old and new rows; another page of its own where there are no such rows.
    first = s["page_table"].gather(1, torch.minimum(before, s["lens"].long() - 1)[:, None] // page)[:, 0].long()
    shared = torch.zeros(cache.shape[0], dtype=torch.bool, device=DEV).index_copy_(0, first, kept > 0)
    written = torch.zeros(cache.shape[0], dtype=torch.bool, device=DEV).index_fill_(0, pid, True)
    least = _least_scale(need)
    fresh = torch.where(shared[:, None], torch.maximum(least, scale), least)
    fresh = torch.where(written[:, None], fresh, scale)
    raw = cache.view(torch.uint8)
    held = raw[first]
    old = (held.view(E4M3).float() * (scale / fresh)[first][..., None, None]).to(E4M3).view(torch.uint8)
    live = (torch.arange(page, device=DEV) < kept[:, None])[:, None, :, None]
    raw[first] = torch.where(live, old, held)
    raw[pid, :, pos % page] = (x / fresh[pid][..., None]).to(E4M3).view(torch.uint8)
    scale.copy_(fresh)


def _append_plain(s):
    b, pos, pid = _places(s)
    k, q = s["k"].float(), s["q"].float()
    if s["inv_freq"] is not None:
        k, q = (_turned(x, pos, s["inv_freq"], s["interleaved"]) for x in (k, q))
    _store(k, s["k_cache"], s["k_scale"], s, b, pos, pid)
    _store(s["v"].float(), s["v_cache"], s["v_scale"], s, b, pos, pid)
    return q.to(torch.bfloat16)


def _gathered(cache, scale, s):
    """[B, H_kv, max_kv, d] in float32; rows past a sequence's length are zero."""
    table = s["page_table"].long().clamp(min=0)
    x = cache.view(torch.uint8)[table].view(E4M3).float() * scale[table][..., None, None]   # [B, pages, H_kv, page, d]
    x = x.transpose(1, 2).flatten(2, 3)[:, :, :s["max_kv"]]
    live = torch.arange(s["max_kv"], device=DEV) < s["lens"][:, None]
    return torch.where(live[:, None, :, None], x, torch.zeros_like(x))


def _paged_plain(s, q):
    T, H, d = q.shape
    H_kv, n = s["H_kv"], s["max_q"]
    n_q, cu = s["cu"][1:] - s["cu"][:-1], s["cu"].long()
    i = torch.arange(n, device=DEV)
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    x = q[rows].float().transpose(1, 2).unflatten(1, (H_kv, -1))                            # [B, H_kv, G, n, d]
    k, v = _gathered(s["k_cache"], s["k_scale"], s), _gathered(s["v_cache"], s["v_scale"], s)
    x = (x.flatten(2, 3) @ k.transpose(-1, -2)).mul_(s["scale"]).unflatten(2, (-1, n))
    end = s["lens"][:, None].expand(-1, n)
    if s["causal"]:
        end = (end - n_q[:, None] + i + 1).clamp(min=0)
    x.masked_fill_(~(torch.arange(s["max_kv"], device=DEV) < end[..., None])[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).unflatten(2, (-1, n)) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + l.log()).squeeze(-1)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = t - cu[b]
    return (o.flatten(1, 2).transpose(1, 2)[b, at].to(torch.bfloat16),
            lse.flatten(1, 2).transpose(1, 2)[b, at].t().contiguous())


# ---------------------------------------------------------------- one pass
def _append_own(fa, s):
    return fa.fa_kv_append(s["k"], s["v"], s["cu"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                           s["page_table"], s["lens"], q=s["q"], inv_freq=s["inv_freq"], interleaved=s["interleaved"])


def _paged_own(fa, s, q):
    return fa.fa_fwd_paged(q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"], s["lens"],
                           s["cu"], scale=s["scale"], causal=s["causal"])


def _updated(s):
    """The cache as its values in units of their page's scale, and the scales."""
    return s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"]


def run(s):
    op = s["op"]
    if own:
        from exact_io_aware_34_gb300 import fa
        if op == "rope":
            out = fa.fa_rope(s["x"], s["positions"], s["inv_freq"], y=s["y"], interleaved=s["interleaved"],
                             transpose=s["transpose"], factor=s["factor"])
            return out if s["y"] is not None else (out,)
        if op == "paged":
            return _paged_own(fa, s, s["q"])
        q = _append_own(fa, s)
        return (q, *_updated(s)) if op == "append" else (*_paged_own(fa, s, q), *_updated(s))
    if op == "rope":
        return _rope_plain(s)
    if op == "paged":
        return _paged_plain(s, s["q"])
    q = _append_plain(s)
    return (q, *_updated(s)) if op == "append" else (*_paged_plain(s, q), *_updated(s))


# ---------------------------------------------------------------- what a pass cannot do without
def _seen(n_q, n_kv, causal):
    """(row, key) pairs of one sequence."""
    if not causal:
        return n_q * n_kv
    return sum(max(0, n_kv - n_q + i + 1) for i in range(n_q))


def work(case):
    d = case["d"]
    if case["op"] == "rope":
        n = case["T"] * (case["heads"] + case["heads_y"])
        return {"bytes": 2 * 2 * n * d + 4 * case["T"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    H, H_kv, page = case["H"], case["H_kv"], case["page"]
    new, lens = _lens(case["new"]), _lens(case["lens"])
    T, B = sum(new), len(new)
    total = {"bytes": 0, "flops": 0}
    if case["op"] != "paged":
        pages = sum(-(-n // page) - (n - k) // page for n, k in zip(lens, new))
        total["bytes"] += T * d * ((2 * 2 * H if case["rot"] else 0) + 2 * 2 * H_kv + 2 * H_kv) + 2 * 4 * pages * H_kv + 4 * pages + 8 * B
        total["flops"] += T * (3 * case["rot"] * (H + H_kv) + 2 * 2 * d * H_kv)
    if case["op"] != "append":
        pages = sum(-(-n // page) for n in lens)
        pairs = sum(_seen(a, b, case["causal"]) for a, b in zip(new, lens))
        total["bytes"] += T * H * (2 * 2 * d + 4) + 2 * sum(lens) * H_kv * d + pages * (4 + 2 * 4 * H_kv) + 8 * B
        total["flops"] += 4 * d * H * pairs
    return total


# ---------------------------------------------------------------- in 64 bits
def _rotate64(x, positions, inv_freq, interleaved, transpose, factor):
    """As complex numbers: each pair times factor * e^{i angle}."""
    half = inv_freq.numel()
    z = x[..., :2 * half].double()
    z = z.unflatten(-1, (half, 2)) if interleaved else z.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.complex(z[..., 0], z[..., 1])
    angle = torch.outer(positions.double(), inv_freq) * (-1.0 if transpose else 1.0)
    z = torch.view_as_real(z * torch.polar(torch.full_like(angle, factor), angle)[:, None])
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., 2 * half:].double()], -1)


def _append64(case, s):
    """(rotated queries, and for K and V what each place of the cache should hold in units of the scale, and the scales)."""
    new, lens, page = _lens(case["new"]), _lens(case["lens"]), case["page"]
    pos = torch.cat([torch.arange(n - k, n, device=DEV) for n, k in zip(lens, new)])
    q, k, v = (s[c].double() for c in ("q", "k", "v"))
    if s["inv_freq"] is not None:
        q, k = (_rotate64(x, pos, s["inv_freq"], case["interleaved"], False, 1.0) for x in (q, k))
    table = s["page_table"].tolist()
    out = [q]
    for x, cache, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        held, scale = cache.float().double(), scale.double().clone()
        t = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            p = n - m
            while p < n:
                end = min(n, (p // page + 1) * page)
                rows, i, a = x[t:t + end - p], table[b][p // page], p % page
                least = [2.0 ** max(LEAST, math.ceil(math.log2(z / TOP))) if z > 0 else 2.0 ** LEAST
                         for z in rows.abs().amax((0, 2)).tolist()]
                to = torch.tensor(least, dtype=torch.float64, device=DEV)
                if a:
                    to = torch.maximum(to, scale[i])
                    held[i, :, :a] *= (scale[i] / to)[:, None, None]
                held[i, :, a:a + end - p] = rows.transpose(0, 1) / to[:, None, None]
                scale[i] = to
                t, p = t + end - p, end
        out += [held, scale]
    return out


def _paged64(case, s, q):
    H_kv, page, d = case["H_kv"], case["page"], case["d"]
    G = case["H"] // H_kv
    new, lens = _lens(case["new"]), _lens(case["lens"])
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros((q.shape[1], q.shape[0]), dtype=torch.float64, device=DEV)
    t = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        ids = s["page_table"][b, :-(-n // page)].long()
        k, v = ((s[c + "_cache"].view(torch.uint8)[ids].view(E4M3).double() * s[c + "_scale"][ids].double()[..., None, None])
                .transpose(0, 1).reshape(H_kv, -1, d)[:, :n] for c in ("k", "v"))
        x = q[t:t + m].double().reshape(m, H_kv, G, d).permute(1, 2, 0, 3)
        x = torch.einsum("hgid,hjd->hgij", x, k) * case["d"] ** -0.5
        if case["causal"]:
            x = x.masked_fill(torch.ones((m, n), dtype=torch.bool, device=DEV).triu(n - m + 1), float("-inf"))
        l = torch.logsumexp(x, -1)
        o[t:t + m] = torch.einsum("hgij,hjd->ihgd", (x - l[..., None]).exp(), v).reshape(m, -1, d)
        lse[:, t:t + m] = l.reshape(-1, m)
        t += m
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_rotate64(x, s["positions"], s["inv_freq"], case["interleaved"], case["transpose"], case["factor"])
                     for x in (s["x"], s["y"]) if x is not None)
    if case["op"] == "paged":
        return _paged64(case, s, s["q"])
    if case["op"] == "append":
        return tuple(_append64(case, s))
    # (The step's attention reads what was rounded to 8 bits before it, which has no value in 64 bits.)
    return (None, None, *_append64(case, s)[1:])
