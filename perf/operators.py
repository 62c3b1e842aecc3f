"""The operators around the attention core, case by case: what is timed and what it is
compared with.

Three operators, each in a plain torch form and as a user of the library calls it:

  modified scores   attention whose scores are capped by a tanh, biased by distance, and
                    masked by documents or a prefix; forward, and forward + backward
  rotary            rotary positions of Q and K (half and interleaved pairs, part of the
                    head, scaled frequencies), and their gradient
  tree              attention of drafted tokens (a tree, or one token) over a paged cache

``own`` False runs the plain form, True the library's calls.
"""
import math
import random

import torch

own = False

MOD, ROT, TREE = "modified scores", "rotary", "tree"


# ------------------------------------------------------------------------------- cases
def _mod(name, B, H, Hkv, Nq, Nk, d, *, causal=True, softcap=0.0, slopes=False, prefix=0,
         doc=0, train=False):
    return {"name": name, "op": MOD, "B": B, "H": H, "Hkv": Hkv, "Nq": Nq, "Nk": Nk, "d": d,
            "causal": causal, "softcap": softcap, "slopes": slopes, "prefix": prefix,
            "doc": doc, "train": train}


def _rot(name, B, H, Hkv, N, d, rot, dtype, *, interleaved=False, factor=1.0, first=0,
         train=False):
    return {"name": name, "op": ROT, "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "rot": rot,
            "dtype": dtype, "interleaved": interleaved, "factor": factor, "first": first,
            "train": train}


def _tree(name, B, H, Hkv, T, length, d, page, *, softcap=0.0):
    return {"name": name, "op": TREE, "B": B, "H": H, "Hkv": Hkv, "T": T, "length": length,
            "d": d, "page": page, "softcap": softcap}


def listed():
    return [
        # a short prompt: latency of one small forward
        _mod("mod_short_d64", 1, 4, 4, 200, 200, 64, softcap=30.0),
        # a long prompt of a capped model with shared key heads
        _mod("mod_prompt_capped_d128", 1, 16, 4, 8192, 8192, 128, softcap=50.0),
        # many documents in one row, as a training set is packed (evaluation of the loss)
        _mod("mod_documents_d64", 2, 16, 16, 4096, 4096, 64, doc=512),
        # a training step's attention, capped scores and shared key heads
        _mod("mod_train_capped_d128", 2, 16, 4, 4096, 4096, 128, softcap=30.0, train=True),
        # a small training step: bidirectional prefix, distance bias, odd length
        _mod("mod_train_prefix_bias_d64", 2, 16, 16, 1000, 1000, 64, slopes=True, prefix=300,
             train=True),
        # long packed training rows with a ragged end
        _mod("mod_train_documents_d128", 1, 8, 8, 10000, 10000, 128, softcap=50.0, doc=1500,
             train=True),
        # one decoded token of a few sequences, far into a scaled context
        _rot("rotary_token", 8, 16, 4, 1, 128, 128, "bf16", factor=4.0, first=100000),
        # a whole prompt, interleaved pairs over half of each head
        _rot("rotary_prompt_interleaved", 2, 16, 4, 8192, 128, 64, "bf16", interleaved=True),
        # a training step's positions in float32: the gradient as well
        _rot("rotary_train_f32", 2, 16, 16, 4096, 64, 64, "f32", train=True),
        # one token of one sequence over a short cache: latency
        _tree("tree_one_token_d64", 1, 16, 16, 1, 1000, 64, 16),
        # a batch of decoded tokens over long caches
        _tree("tree_batch_d128", 32, 16, 4, 1, 8192, 128, 64),
        # drafted trees over very long caches, capped scores
        _tree("tree_drafts_capped_d128", 8, 16, 2, 32, 32768, 128, 128, softcap=50.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice([MOD, MOD, ROT, TREE])
    if op == MOD:
        train = rng.random() < 0.5
        Hkv = rng.choice([2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4])
        B = rng.choice([1, 2])
        Nk = _log_int(rng, 150, int(2900 * min(1.0, 32 / (B * H)) ** 0.5))
        causal = rng.random() < 0.8
        doc = rng.choice([0, 0, max(150, Nk // 5)])
        Nq = Nk if rng.random() < 0.7 else max(100, int(Nk * rng.uniform(0.2, 0.9)))
        return _mod("", B, H, Hkv, Nq, Nk, rng.choice([64, 128]), causal=causal,
                    softcap=rng.choice([0.0, 20.0, 50.0]), slopes=rng.random() < 0.3,
                    prefix=rng.choice([0, int(Nk * rng.uniform(0.05, 0.9))]) if causal else 0,
                    doc=doc, train=train)
    if op == ROT:
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        return _rot("", rng.choice([1, 2, 3]), Hkv * rng.choice([1, 2, 4]), Hkv,
                    _log_int(rng, 1, 8192), d, rng.choice([d, d // 2, d // 4, d - 4]),
                    rng.choice(["bf16", "bf16", "f32"]), interleaved=rng.random() < 0.5,
                    factor=rng.choice([1.0, 4.0, 8.0]), first=_log_int(rng, 1, 200000),
                    train=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    T = rng.choice([1, 1, rng.randint(2, 64)])
    B = _log_int(rng, 1, 32)
    return _tree("", B, Hkv * rng.choice([1, 2, 4, 8]), Hkv, T,
                 _log_int(rng, 70, min(100000, 2 ** 20 // (B * Hkv))), rng.choice([64, 128]),
                 rng.choice([16, 32, 64, 128]), softcap=rng.choice([0.0, 0.0, 30.0]))


# -------------------------------------------------------- sizes that follow from a case
def _documents(case):
    """Document lengths of each row (they fill the row but for a few padding tokens)."""
    rows = []
    for b in range(case["B"]):
        rng = random.Random(f"{case['Nk']} {case['doc']} {b}")
        left, lens = case["Nk"] - (b * 37) % 64, []
        while left > 0:
            n = min(left, max(1, int(case["doc"] * rng.uniform(0.3, 1.7))))
            lens.append(n)
            left -= n
        rows.append(lens)
    return rows


def _lengths(case):
    """Cached tokens of each sequence, drafted ones included."""
    rng = random.Random(f"{case['B']} {case['length']} {case['T']}")
    L = case["length"]
    return [max(case["T"], L if b == 0 else int(L * rng.uniform(0.6, 1.0)))
            for b in range(case["B"])]


def _limits(case, b):
    """First and one past the last visible key of every query row of sequence b."""
    Nq, Nk = case["Nq"], case["Nk"]
    p = torch.arange(Nk - Nq, Nk)
    lo, hi = torch.zeros(Nq, dtype=torch.int64), torch.full((Nq,), Nk)
    if case["causal"]:
        hi = (p + 1).clamp(min=min(case["prefix"], Nk))
    if case["doc"]:
        start, end = torch.arange(Nk), torch.arange(Nk)  # padding: nothing
        at = 0
        for n in _documents(case)[b]:
            start[at:at + n], end[at:at + n] = at, at + n
            at += n
        inside = p >= 0  # a query in front of the first key is in no document
        at = p.clamp(min=0)
        lo = torch.where(inside, start[at], 0)
        hi = torch.minimum(hi, torch.where(inside, end[at], 0))
    return lo, torch.maximum(hi, lo)


def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == MOD:
        pairs = case["H"] * sum(int((hi - lo).sum()) for lo, hi in
                                (_limits(case, b) for b in range(case["B"])))
        q = case["B"] * case["H"] * case["Nq"] * case["d"] * 2
        kv = case["B"] * case["Hkv"] * case["Nk"] * case["d"] * 2
        lse = case["B"] * case["H"] * case["Nq"] * 4
        by = 2 * q + 2 * kv + lse
        if case["train"]:
            return {"bytes": by + q * 2 + 2 * kv, "flops": 14 * case["d"] * pairs}
        return {"bytes": by, "flops": 4 * case["d"] * pairs}
    if case["op"] == ROT:
        rows = case["B"] * case["N"] * (case["H"] + case["Hkv"])
        n = 2 if case["train"] else 1
        return {"bytes": n * 2 * rows * case["d"] * e, "flops": n * 3 * rows * case["rot"]}
    tokens = sum(_lengths(case))
    q = case["B"] * case["H"] * case["T"] * case["d"] * 2
    return {"bytes": 2 * tokens * case["Hkv"] * case["d"] * 2 + 2 * q + q * 2 // case["d"],
            "flops": 4 * case["d"] * tokens * case["H"] * case["T"]}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, sigma=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)

    s = dict(case)
    B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
    if case["op"] == MOD:
        # queries and keys a little wider than unit: the cap then bends the largest scores
        s["Q"] = normal(B, H, case["Nq"], d, sigma=1.5)
        s["K"] = normal(B, Hkv, case["Nk"], d, sigma=1.5)
        s["V"] = normal(B, Hkv, case["Nk"], d)
        s["dO"] = normal(B, H, case["Nq"], d) if case["train"] else None
        s["slope"] = None
        if case["slopes"]:
            # the usual geometric series over the heads
            s["slope"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda") / H)
        s["prefix_len"] = None
        if case["prefix"]:
            s["prefix_len"] = torch.full((B,), case["prefix"], dtype=torch.int32, device="cuda")
        s["doc_ids"] = None
        if case["doc"]:
            ids = torch.full((B, case["Nk"]), -1, dtype=torch.int32)
            for b, lens in enumerate(_documents(case)):
                row = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
                ids[b, :len(row)] = row.int()
            s["doc_ids"] = ids.cuda()
    elif case["op"] == ROT:
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["Q"], s["K"] = normal(B, H, case["N"], d, dtype=dt), normal(B, Hkv, case["N"], d, dtype=dt)
        if case["train"]:
            s["dQ"] = normal(B, H, case["N"], d, dtype=dt)
            s["dK"] = normal(B, Hkv, case["N"], d, dtype=dt)
        k = torch.arange(case["rot"] // 2, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2 * k / case["rot"]) / case["factor"]).float().cuda()
        s["mscale"] = 0.1 * math.log(case["factor"]) + 1.0
        start = torch.randint(0, case["first"] + 1, (B, 1), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(case["N"], device="cuda")).int()
    else:
        T, page = case["T"], case["page"]
        lens = _lengths(case)
        pages = [-(-n // page) for n in lens]
        total = sum(pages) + 3
        s["Q"] = normal(B, H, T, d, sigma=1.5)
        s["K"] = normal(total, Hkv, page, d, sigma=1.5)
        s["V"] = normal(total, Hkv, page, d)
        ids = torch.randperm(total, generator=g, device="cuda").int()
        s["table"] = torch.zeros(B, max(pages), dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            s["table"][b, :n] = ids[at:at + n]
            at += n
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["bits"] = None
        if T > 1:
            # every drafted token hangs below one of the tokens drafted before it
            rng, rows = random.Random(seed), []
            for b in range(B):
                bits = [1]
                for t in range(1, T):
                    bits.append(bits[rng.randrange(max(0, t - 8), t)] | 1 << t)
                rows.append([x - (1 << 64) if x >> 63 else x for x in bits])
            s["bits"] = torch.tensor(rows, dtype=torch.int64, device="cuda")
    return s


# ---------------------------------------------------------------------- the plain forms
def _mod_plain(s):
    B, H, Hkv, Nq, Nk, d = (s[n] for n in ("B", "H", "Hkv", "Nq", "Nk", "d"))
    G = H // Hkv
    scale = 1.0 / math.sqrt(d)
    q = s["Q"].float().view(B, Hkv, G, Nq, d)
    k, v = s["K"].float()[:, :, None], s["V"].float()[:, :, None]
    x = torch.matmul(q, k.transpose(-1, -2)) * scale
    t = None
    if s["softcap"]:
        t = torch.tanh(x / s["softcap"])
        x = t * s["softcap"]
    p = torch.arange(Nk - Nq, Nk, device=x.device)[:, None]
    j = torch.arange(Nk, device=x.device)[None, :]
    if s["slope"] is not None:
        x = x - s["slope"].view(Hkv, G, 1, 1) * (p - j).abs().float()
    seen = torch.ones(B, Nq, Nk, dtype=torch.bool, device=x.device)
    if s["causal"]:
        seen = seen & (j <= p)
        if s["prefix_len"] is not None:
            seen = seen | (j < s["prefix_len"][:, None, None])
    if s["doc_ids"] is not None:
        ids = s["doc_ids"]
        mine = torch.where(p[:, 0] >= 0, ids[:, p[:, 0].clamp(min=0)], -1)
        seen = seen & (mine[:, :, None] == ids[:, None, :]) & (ids[:, None, :] >= 0)
    seen = seen[:, None, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    P = e / torch.where(l == 0, 1.0, l)
    O = torch.matmul(P, v)
    out = {"O": O.view(B, H, Nq, d).to(s["Q"].dtype),
           "LSE": (m + torch.log(l)).view(B, H, Nq)}
    if s["train"]:
        g = s["dO"].float().view(B, Hkv, G, Nq, d)
        dV = torch.matmul(P.transpose(-1, -2), g).sum(2)
        dS = torch.matmul(g, v.transpose(-1, -2))
        dS = P * (dS - (g * O).sum(-1, keepdim=True))
        if t is not None:
            dS = dS * (1 - t * t)
        out["dQ"] = (torch.matmul(dS, k) * scale).view(B, H, Nq, d).to(s["Q"].dtype)
        out["dK"] = (torch.matmul(dS.transpose(-1, -2), q).sum(2) * scale).to(s["K"].dtype)
        out["dV"] = dV.to(s["V"].dtype)
    return out


def _turn(x, s, sign):
    ang = s["positions"].double()[:, None, :, None] * s["inv_freq"].double()
    c, sn = (ang.cos() * s["mscale"]).float(), (ang.sin() * (s["mscale"] * sign)).float()
    R = s["rot"]
    y = x.float()
    if s["interleaved"]:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        r = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        r = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((r, y[..., R:]), -1).to(x.dtype)


def _rot_plain(s):
    out = {"Q": _turn(s["Q"], s, 1.0), "K": _turn(s["K"], s, 1.0)}
    if s["train"]:
        out["dQ"], out["dK"] = _turn(s["dQ"], s, -1.0), _turn(s["dK"], s, -1.0)
    return out


def _tree_plain(s):
    B, H, Hkv, T, d = (s[n] for n in ("B", "H", "Hkv", "T", "d"))
    G = H // Hkv
    k = s["K"][s["table"].long()].float().transpose(1, 2).reshape(B, Hkv, -1, d)
    v = s["V"][s["table"].long()].float().transpose(1, 2).reshape(B, Hkv, -1, d)
    q = s["Q"].float().view(B, Hkv, G * T, d)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    if s["softcap"]:
        x = torch.tanh(x / s["softcap"]) * s["softcap"]
    j = torch.arange(k.shape[2], device=x.device)
    u = j[None, :] - (s["lens"][:, None] - T)  # number of a key among the drafted tokens
    seen = (u < 0)[:, None, :].expand(B, T, -1)
    drafted = ((u >= 0) & (u < T))[:, None, :]
    if s["bits"] is None:
        seen = seen | drafted
    else:
        seen = seen | drafted & ((s["bits"][:, :, None] >> u.clamp(0, 63)[:, None, :]) & 1).bool()
    x = x.view(B, Hkv, G, T, -1)
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    O = torch.matmul((e / l).view(B, Hkv, G * T, -1), v)
    return {"O": O.view(B, H, T, d).to(s["Q"].dtype), "LSE": (m + torch.log(l)).view(B, H, T)}


# ------------------------------------------------------------------------------ one pass
def run(s):
    if not own:
        if s["op"] == MOD:
            return _mod_plain(s)
        return _rot_plain(s) if s["op"] == ROT else _tree_plain(s)
    from exact_io_aware_64_b200 import binding
    if s["op"] == MOD:
        docs = binding.doc_ranges(s["doc_ids"]) if s["doc_ids"] is not None else None
        mod = {"causal": s["causal"], "softcap": s["softcap"], "slopes": s["slope"],
               "prefix": s["prefix_len"], "docs": docs}
        O, LSE = binding.fwd_mod(s["Q"], s["K"], s["V"], **mod)
        out = {"O": O, "LSE": LSE}
        if s["train"]:
            out["dQ"], out["dK"], out["dV"] = binding.bwd_mod(s["Q"], s["K"], s["V"], O, s["dO"],
                                                              LSE, **mod)
        return out
    if s["op"] == ROT:
        how = {"positions": s["positions"], "interleaved": s["interleaved"],
               "mscale": s["mscale"]}
        q, k = binding.rotary(s["Q"], s["K"], s["inv_freq"], **how)
        out = {"Q": q, "K": k}
        if s["train"]:
            out["dQ"], out["dK"] = binding.rotary_bwd(s["dQ"], s["dK"], s["inv_freq"], **how)
        return out
    O, LSE = binding.fwd_tree(s["Q"], s["K"], s["V"], s["table"], s["lens"],
                              tree_mask=s["bits"], softcap=s["softcap"])
    return {"O": O, "LSE": LSE}


# ------------------------------------------------------------- the definition in 64 bits
def _exact_head(q, k, v, lo, hi, scale, cap, slope, p0, dO=None):
    """One query head, rows in blocks: softmax over the keys lo[i] <= j < hi[i]."""
    Nq, Nk = q.shape[0], k.shape[0]
    j = torch.arange(Nk, device=q.device)
    O = torch.zeros(Nq, v.shape[1], dtype=torch.float64, device=q.device)
    L = torch.full((Nq,), -math.inf, dtype=torch.float64, device=q.device)
    dQ, dK, dV = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for r in range(0, Nq, 2048):
        R = slice(r, min(r + 2048, Nq))
        z = torch.einsum("id,jd->ij", q[R], k) * scale
        grad = 1.0
        if cap:
            th = torch.tanh(z / cap)
            z, grad = cap * th, 1.0 / torch.cosh(z / cap) ** 2
        if slope is not None:
            i = torch.arange(R.start, R.stop, device=q.device) + p0
            z = z - slope * (i[:, None] - j).abs()
        hidden = (j[None, :] < lo[R, None]) | (j[None, :] >= hi[R, None])
        z = z.masked_fill(hidden, -math.inf)
        L[R] = torch.logsumexp(z, 1)
        P = torch.exp(z - torch.where(L[R] == -math.inf, 0.0, L[R])[:, None])
        O[R] = P @ v
        if dO is not None:
            dP = dO[R] @ v.T
            dZ = P * (dP - (P * dP).sum(1, keepdim=True)) * grad
            dQ[R] = scale * (dZ @ k)
            dK += scale * (dZ.T @ q[R])
            dV += P.T @ dO[R]
    return O, L, dQ, dK, dV


def _exact_mod(case, s):
    B, H, Hkv = case["B"], case["H"], case["Hkv"]
    out = {"O": torch.zeros_like(s["Q"], dtype=torch.float64),
           "LSE": torch.zeros(B, H, case["Nq"], dtype=torch.float64, device="cuda")}
    if case["train"]:
        out["dQ"] = torch.zeros_like(s["Q"], dtype=torch.float64)
        out["dK"] = torch.zeros_like(s["K"], dtype=torch.float64)
        out["dV"] = torch.zeros_like(s["V"], dtype=torch.float64)
    for b in range(B):
        lo, hi = (x.cuda() for x in _limits(case, b))
        for h in range(H):
            c = h // (H // Hkv)
            got = _exact_head(s["Q"][b, h].double(), s["K"][b, c].double(), s["V"][b, c].double(),
                              lo, hi, case["d"] ** -0.5, case["softcap"],
                              s["slope"][h].double() if case["slopes"] else None,
                              case["Nk"] - case["Nq"],
                              s["dO"][b, h].double() if case["train"] else None)
            out["O"][b, h], out["LSE"][b, h] = got[0], got[1]
            if case["train"]:
                out["dQ"][b, h] = got[2]
                out["dK"][b, c] += got[3]
                out["dV"][b, c] += got[4]
    return out


def _exact_rot(case, s):
    R = case["rot"]

    def turned(x, sign):
        first = torch.arange(R // 2, device="cuda")
        a, b = (2 * first, 2 * first + 1) if case["interleaved"] else (first, first + R // 2)
        ang = sign * torch.einsum("bn,k->bnk", s["positions"].double(), s["inv_freq"].double())
        w = torch.polar(torch.full_like(ang, s["mscale"]), ang)[:, None]
        x = x.double()
        z = torch.complex(x[..., a], x[..., b]) * w
        y = x.clone()
        y[..., a], y[..., b] = z.real, z.imag
        return y

    out = {"Q": turned(s["Q"], 1), "K": turned(s["K"], 1)}
    if case["train"]:
        out["dQ"], out["dK"] = turned(s["dQ"], -1), turned(s["dK"], -1)
    return out


def _exact_tree(case, s):
    B, H, Hkv, T, d, page = (case[n] for n in ("B", "H", "Hkv", "T", "d", "page"))
    O = torch.zeros(B, H, T, d, dtype=torch.float64, device="cuda")
    L = torch.zeros(B, H, T, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        at = torch.arange(n, device="cuda")
        pg = s["table"][b].long()[at // page]
        seen = torch.ones(T, n, dtype=torch.bool, device="cuda")
        if s["bits"] is not None:
            bits = s["bits"][b].tolist()
            seen[:, n - T:] = torch.tensor([[bool(x >> u & 1) for u in range(T)] for x in bits])
        for h in range(H):
            c = h // (H // Hkv)
            k, v = s["K"][pg, c, at % page].double(), s["V"][pg, c, at % page].double()
            z = s["Q"][b, h].double() @ k.T * d ** -0.5
            if case["softcap"]:
                z = case["softcap"] * torch.tanh(z / case["softcap"])
            z = z.masked_fill(~seen, -math.inf)
            L[b, h] = torch.logsumexp(z, 1)
            O[b, h] = torch.exp(z - L[b, h][:, None]) @ v
    return {"O": O, "LSE": L}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == MOD:
        return _exact_mod(case, s)
    return _exact_rot(case, s) if case["op"] == ROT else _exact_tree(case, s)
