"""Workloads of the attention side of a decoder block, next to its sparse FFN:

``append``     writing a step's keys and values into a paged cache, the heads of
               q and k normalised and rotated by position on the way
``attention``  attention of each sequence's new tokens over its paged cache
``norm``       RMS norm and position rotation of q and k for training, forward
``norm_grad``  and its gradients: q, k and both norm weights

``listed`` and ``draw`` give cases, ``prepare`` what a program holds before a
call, ``run`` one call: in plain torch operations in 32 bits, or (``own``)
through the library.  ``exact`` is the same result from the definition in 64
bits, ``work`` the bytes and operations that a call cannot do without.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ the cases
def _attention(name, mix, n_seqs, max_q, max_kv, hq, hkv, dim, page, window=0, causal=True,
               dtype="bf16"):
    return {"name": name, "op": "attention", "mix": mix, "n_seqs": n_seqs, "max_q": max_q,
            "max_kv": max_kv, "hq": hq, "hkv": hkv, "dim": dim, "page": page, "window": window,
            "causal": causal, "dtype": dtype}


def _heads(name, op, tokens, hq, hkv, dim, rot, norm=True, adjacent=False, dtype="bf16", page=0,
           skip=0):
    return {"name": name, "op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim, "rot": rot,
            "norm": norm, "adjacent": adjacent, "dtype": dtype, "page": page, "skip": skip}


def listed():
    return [
        # one user, one token: latency of a short context
        _attention("attention_decode_one", 1, 1, 1, 257, 16, 4, 128, 16),
        # a decode batch of 32 (width 4096) with contexts of all lengths
        _attention("attention_decode_batch", 2, 32, 1, 4096, 32, 8, 128, 16),
        # a few users with very long contexts: the cache is read once
        _attention("attention_decode_long", 3, 3, 1, 131000, 32, 8, 128, 64),
        # drafts of up to five tokens checked at once, sliding window, narrow heads
        _attention("attention_verify_window", 4, 24, 5, 8000, 32, 4, 64, 32, window=1000),
        # prompts prefilled in chunks while other users decode, one batch
        _attention("attention_mixed", 5, 12, 1024, 12000, 32, 8, 128, 32),
        # a whole prompt of the large workload's length
        _attention("attention_prompt", 6, 1, 16384, 16384, 32, 8, 128, 64),
        # float32, odd head width, pages that no tile divides, ragged chunks
        _attention("attention_f32", 7, 5, 333, 2100, 8, 8, 80, 24, dtype="f32"),
        # a decode step of 32 tokens
        _heads("append_decode", "append", 32, 32, 8, 128, 128, page=16),
        # a prompt of 16384 tokens, some of them padding that is not stored
        _heads("append_prompt", "append", 16384, 32, 8, 128, 128, norm=False, page=64, skip=37),
        # training: 16384 tokens a step, forward and backward
        _heads("norm_train", "norm", 16384, 32, 8, 128, 128),
        _heads("norm_grad_train", "norm_grad", 16384, 32, 8, 128, 128),
        # a small float32 step whose heads are rotated in part, pairs side by side
        _heads("norm_grad_f32", "norm_grad", 1001, 16, 4, 80, 40, adjacent=True, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    while True:
        case = _draw(rng)
        cost = work(case)
        # float32 products run at a sixteenth of the bfloat16 rate
        flops = cost["flops"] * (16 if case["dtype"] == "f32" else 1)
        if cost["bytes"] < 9e8 and flops < 2e12:
            return case


def _draw(rng):
    op = rng.choice(["attention"] * 5 + ["append"] * 2 + ["norm"] + ["norm_grad"] * 2)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hq, hkv = rng.choice([(32, 8), (16, 16), (16, 4), (8, 1), (28, 4), (40, 8), (5, 5)])
    dim = rng.choice([64, 80, 128, 128, 128, 256])
    if op != "attention":
        rot = rng.choice([dim, dim, dim // 2])
        page = rng.choice([1, 16, 24, 64, 256]) if op == "append" else 0
        tokens = _log(rng, 1, 16384 * 32 * 128 // (hq * dim) if dtype == "bf16" else 4000)
        tokens = min(tokens, 16384)
        return _heads(None, op, tokens, hq, hkv, dim, rot, rng.random() < 0.7 or op == "norm_grad",
                      rng.random() < 0.3, dtype, page,
                      rng.choice([0, 5, 37]) if op == "append" else 0)
    kind = rng.choice(["decode", "decode", "few", "chunk", "prompt"])
    mix, page = rng.randrange(1 << 30), rng.choice([1, 16, 24, 64, 256])
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    if kind == "prompt":
        n_seqs, max_q = rng.choice([1, 2, 3]), _log(rng, 2, 4500)
        max_kv = max_q
    elif kind == "chunk":
        n_seqs, max_q = _log(rng, 1, 12), _log(rng, 32, 700)
        max_kv = max_q + _log(rng, 1, 9000)
    else:
        n_seqs, max_q = _log(rng, 1, 96), 1 if kind == "decode" else rng.randrange(2, 10)
        max_kv = max_q + _log(rng, 1, max(2, min(120000, 300000 // n_seqs)))
    return _attention(None, mix, n_seqs, max_q, max_kv, hq, hkv, dim, page, window,
                      rng.random() < 0.9, dtype)


def _lengths(case):
    """New tokens and cached length (those included) of every sequence."""
    rng = random.Random(case["mix"])
    q, kv = [case["max_q"]], [case["max_kv"]]
    for _ in range(case["n_seqs"] - 1):
        n = 1 if case["max_q"] == 1 or rng.random() < 0.3 else rng.randint(1, case["max_q"])
        q.append(n)
        kv.append(rng.randint(n, case["max_kv"]))
    order = list(range(case["n_seqs"]))
    rng.shuffle(order)
    return [q[i] for i in order], [kv[i] for i in order]


# ------------------------------------------------------------------ the inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _table(rows, rot):
    """cos | sin of every position, [rows, rot] float32."""
    freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq[None, :]
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def _prepare_attention(case, gen):
    q_len, kv_len = _lengths(case)
    tokens, dim, page, dt = sum(q_len), case["dim"], case["page"], _dtype(case)
    pages = [-(-n // page) for n in kv_len]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(kv_len), max(pages)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in q_len:
        starts.append(starts[-1] + n)
    s = {"case": case, "q_len": q_len, "kv_len_host": kv_len,
         "q": _normal(gen, (tokens, case["hq"], dim), dt),
         "k_cache": _normal(gen, (n_pages, page, case["hkv"], dim), dt),
         "v_cache": _normal(gen, (n_pages, page, case["hkv"], dim), dt),
         "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
         "block_table": table}
    if own:
        from activation_sparse_feed_amd import sffn
        s["batch"] = sffn.make_paged_batch(
            tokens, len(kv_len), case["hq"], case["hkv"], dim, dt, page, n_pages, max(pages),
            max(q_len), max(kv_len), causal=case["causal"], window=case["window"])
        s["workspace"] = sffn.alloc_paged_workspace(s["batch"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((tokens, case["hq"]), dtype=torch.float32, device="cuda")
    return s


def _prepare_heads(case, gen):
    n, hq, hkv, dim, dt = case["tokens"], case["hq"], case["hkv"], case["dim"], _dtype(case)
    # the projection's output: q, k and v side by side in one row of each token
    qkv = _normal(gen, (n, hq + 2 * hkv, dim), dt)
    max_pos = max(2 * n, 4096)
    s = {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
         "q_weight": None, "k_weight": None, "table": _table(max_pos, case["rot"]),
         "positions": torch.randint(0, max_pos, (n,), generator=gen, device="cuda").to(torch.int32)}
    if case["norm"]:
        s["q_weight"] = (1 + _normal(gen, (dim,), torch.float32, 0.2)).to(dt)
        s["k_weight"] = (1 + _normal(gen, (dim,), torch.float32, 0.2)).to(dt)
    if case["op"] == "append":
        page = case["page"]
        n_pages = -(-n // page) + 5
        slots = torch.randperm(n_pages, generator=gen, device="cuda")[:, None] * page
        slots = (slots + torch.arange(page, device="cuda")[None, :]).reshape(-1)[:n].to(torch.int32)
        if case["skip"]:
            slots[case["skip"] - 1::case["skip"]] = -1  # padding tokens are not stored
        s["slots"] = slots
        s["k_cache"] = _normal(gen, (n_pages, page, hkv, dim), dt)
        s["v_cache"] = _normal(gen, (n_pages, page, hkv, dim), dt)
    if case["op"] == "norm_grad":
        s["gq_out"] = _normal(gen, (n, hq, dim), dt)
        s["gk_out"] = _normal(gen, (n, hkv, dim), dt)
    if own:
        from activation_sparse_feed_amd import sffn
        s["heads"] = sffn.make_heads(n, hq, hkv, dim, dt, rot_dim=case["rot"], max_pos=max_pos,
                                     norm=case["norm"], eps=EPS, adjacent=case["adjacent"])
        s["q_out"] = torch.empty((n, hq, dim), dtype=dt, device="cuda")
        if case["op"] != "append":
            s["k_out"] = torch.empty((n, hkv, dim), dtype=dt, device="cuda")
        if case["op"] == "norm_grad":
            s["gq_weight"] = torch.empty(dim, dtype=torch.float32, device="cuda")
            s["gk_weight"] = torch.empty(dim, dtype=torch.float32, device="cuda")
            s["workspace"] = sffn.alloc_heads_workspace(s["heads"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (_prepare_attention if case["op"] == "attention" else _prepare_heads)(case, gen)


# ------------------------------------------------- one call through the library
def _run_own(s):
    from activation_sparse_feed_amd import sffn
    op = s["case"]["op"]
    if op == "attention":
        sffn.paged_attn_fwd(s["batch"], s["q"], s["k_cache"], s["v_cache"], s["q_start"],
                            s["kv_len"], s["block_table"], s["out"], s["workspace"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "append":
        sffn.paged_kv_append(s["heads"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"],
                             s["table"], s["positions"], s["slots"], s["q_out"], s["k_cache"],
                             s["v_cache"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "norm":
        sffn.qk_norm_rope(s["heads"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"],
                          s["positions"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    sffn.qk_norm_rope_bwd(s["heads"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["table"],
                          s["positions"], s["gq_out"], s["gk_out"], s["q_out"], s["k_out"],
                          s["gq_weight"], s["gk_weight"], s["workspace"])
    return s["q_out"], s["k_out"], s["gq_weight"], s["gk_weight"]


# ------------------------------------------------------- the plain form, 32 bits
def _plain_attention(s):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    g, scale, dt = hq // hkv, 1.0 / math.sqrt(dim), _dtype(case)
    out = torch.empty_like(s["q"])
    lse = torch.empty((s["q"].shape[0], hq), dtype=torch.float32, device="cuda")
    at = 0
    for i, (nq, nkv) in enumerate(zip(s["q_len"], s["kv_len_host"])):
        pages = s["block_table"][i, :-(-nkv // case["page"])].long()
        lo = max(0, nkv - nq - case["window"] + 1) if case["window"] else 0
        k = s["k_cache"][pages].reshape(-1, hkv, dim)[lo:nkv].float().permute(1, 2, 0).contiguous()
        v = s["v_cache"][pages].reshape(-1, hkv, dim)[lo:nkv].float().permute(1, 0, 2).contiguous()
        cols = torch.arange(lo, nkv, device="cuda")
        # rows in blocks, so that the scores fit
        step = max(1, min(nq, (1 << 30) // (hq * max(1, nkv - lo))))
        for r in range(0, nq, step):
            n = min(step, nq - r)
            q = s["q"][at + r:at + r + n].float().reshape(n, hkv, g, dim).permute(1, 0, 2, 3)
            p = torch.matmul(q.reshape(hkv, n * g, dim), k).mul_(scale).view(hkv, n, g, nkv - lo)
            pos = torch.arange(nkv - nq + r, nkv - nq + r + n, device="cuda")[:, None]
            if case["causal"] or case["window"]:
                hide = torch.zeros((n, nkv - lo), dtype=torch.bool, device="cuda")
                if case["causal"]:
                    hide |= cols[None, :] > pos
                if case["window"]:
                    hide |= cols[None, :] <= pos - case["window"]
                p.masked_fill_(hide[None, :, None, :], -math.inf)
            top = p.amax(-1, keepdim=True)
            p.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(hkv, n * g, nkv - lo), v).view(hkv, n, g, dim) / total
            out[at + r:at + r + n] = o.permute(1, 0, 2, 3).reshape(n, hq, dim).to(dt)
            lse[at + r:at + r + n] = (top + total.log()).permute(1, 0, 2, 3).reshape(n, hq)
            del p, q, o
        at += nq
    return out, lse


def _pairs(x, rot, adjacent):
    """The two members of every rotated pair, and what is not rotated."""
    if adjacent:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, adjacent):
    if adjacent:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _angles(s):
    rot = s["case"]["rot"]
    rows = s["table"][s["positions"].long()][:, None, :]
    return rows[..., :rot // 2], rows[..., rot // 2:]


def _plain_rotated(s, x, weight):
    case = s["case"]
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    c, z = _angles(s)
    a, b, rest = _pairs(x, case["rot"], case["adjacent"])
    return _join(a * c - b * z, b * c + a * z, rest, case["adjacent"]).to(_dtype(case))


def _plain_grad(s, x, weight, gy):
    case = s["case"]
    x, gy = x.float(), gy.float()
    c, z = _angles(s)
    a, b, rest = _pairs(gy, case["rot"], case["adjacent"])
    gn = _join(a * c + b * z, b * c - a * z, rest, case["adjacent"])
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    gw = (gn * xh).sum((0, 1))
    gh = gn * weight.float()
    gx = r * (gh - xh * (gh * xh).mean(-1, keepdim=True))
    return gx.to(_dtype(case)), gw


def _run_plain(s):
    op = s["case"]["op"]
    if op == "attention":
        return _plain_attention(s)
    if op == "norm_grad":
        gq, gqw = _plain_grad(s, s["q"], s["q_weight"], s["gq_out"])
        gk, gkw = _plain_grad(s, s["k"], s["k_weight"], s["gk_out"])
        return gq, gk, gqw, gkw
    q, k = _plain_rotated(s, s["q"], s["q_weight"]), _plain_rotated(s, s["k"], s["k_weight"])
    if op == "norm":
        return q, k
    slots, v = s["slots"].long(), s["v"]
    if s["case"]["skip"]:
        keep = (slots >= 0).nonzero()[:, 0]
        slots, k, v = slots[keep], k[keep], v[keep]
    s["k_cache"].view(-1, *k.shape[1:])[slots] = k
    s["v_cache"].view(-1, *v.shape[1:])[slots] = v
    return q, s["k_cache"], s["v_cache"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------- the definition in 64 bits
def _exact_attention(s):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    slot_of = torch.arange(max(s["kv_len_host"]), device="cuda")
    at = 0
    for i, (nq, nkv) in enumerate(zip(s["q_len"], s["kv_len_host"])):
        j = slot_of[:nkv]
        page = s["block_table"][i].long()[j // case["page"]]
        pos = torch.arange(nq, device="cuda")[:, None] + (nkv - nq)
        seen = torch.ones((nq, nkv), dtype=torch.bool, device="cuda")
        if case["causal"]:
            seen &= j[None, :] <= pos
        if case["window"]:
            seen &= pos - j[None, :] < case["window"]
        for h in range(hkv):
            k = s["k_cache"][page, j % case["page"], h].double()
            v = s["v_cache"][page, j % case["page"], h].double()
            for head in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                for r in range(0, nq, 4096):
                    e = min(nq, r + 4096)
                    z = s["q"][at + r:at + e, head].double() @ k.T.contiguous() / math.sqrt(dim)
                    z = torch.where(seen[r:e], z, -math.inf)
                    lse[at + r:at + e, head] = torch.logsumexp(z, -1)
                    out[at + r:at + e, head] = torch.softmax(z, -1) @ v
        at += nq
    return out, lse


def _exact_rotated(s, x, weight):
    case = s["case"]
    rot, dim = case["rot"], case["dim"]
    if case["norm"]:
        x = x / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / dim + EPS) * weight
    row = s["table"].double()[s["positions"].long()]
    # every rotated element gets cos * itself + sign * sin * its partner
    e = torch.arange(rot, device="cuda")
    if case["adjacent"]:
        pair, partner, sign = e // 2, e ^ 1, torch.where(e % 2 == 0, -1.0, 1.0).double()
    else:
        pair, partner = e % (rot // 2), (e + rot // 2) % rot
        sign = torch.where(e < rot // 2, -1.0, 1.0).double()
    c, z = row[:, pair][:, None, :], (row[:, rot // 2 + pair] * sign)[:, None, :]
    return torch.cat([x[..., :rot] * c + x[..., partner] * z, x[..., rot:]], -1)


def exact(case, seed):
    if case["op"] == "attention":
        q_len, kv_len = _lengths(case)
        # about 20 seconds: launches of the loops over heads, and products
        pairs = sum(a * b for a, b in zip(q_len, kv_len)) * case["hq"]
        if len(q_len) * case["hq"] > 8000 or pairs * case["dim"] > 1.5e12:
            return None
        return _exact_attention(prepare(case, seed))
    s = prepare(case, seed)
    x = {n: s[n].double() for n in ("q", "k")}
    w = {n: s[n + "_weight"].double() if case["norm"] else None for n in ("q", "k")}
    if case["op"] == "norm_grad":
        res = {}
        for n in ("q", "k"):
            xi, wi = x[n].requires_grad_(True), w[n].requires_grad_(True)
            y = _exact_rotated(s, xi, wi)
            res[n] = torch.autograd.grad(y, (xi, wi), s["g" + n + "_out"].double())
        return res["q"][0], res["k"][0], res["q"][1], res["k"][1]
    with torch.no_grad():
        q, k = _exact_rotated(s, x["q"], w["q"]), _exact_rotated(s, x["k"], w["k"])
    if case["op"] == "norm":
        return q, k
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    t = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][t].long()
    kc[slot // case["page"], slot % case["page"]] = k[t]
    vc[slot // case["page"], slot % case["page"]] = s["v"][t].double()
    return q, kc, vc


# -------------------------------------------- what a call cannot do without
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if case["op"] == "attention":
        q_len, kv_len = _lengths(case)
        pairs = keys = 0
        for nq, nkv in zip(q_len, kv_len):
            keys += min(nkv, nq + case["window"] - 1) if case["window"] else nkv
            for pos in range(nkv - nq, nkv):
                end = pos + 1 if case["causal"] else nkv
                pairs += end - max(0, pos - case["window"] + 1) if case["window"] else end
        tokens = sum(q_len)
        table = sum(-(-n // case["page"]) for n in kv_len) * 4 + 8 * len(kv_len) + 4
        return {"bytes": 2 * tokens * hq * dim * size + 4 * tokens * hq +
                2 * keys * hkv * dim * size + table, "flops": 4 * pairs * hq * dim}
    n, rows = case["tokens"], case["tokens"] * (hq + hkv)
    angles = 4 * n + min(n, max(2 * n, 4096)) * case["rot"] * 4
    weights = 2 * dim * size if case["norm"] else 0
    if case["op"] == "norm_grad":
        return {"bytes": 3 * rows * dim * size + angles + weights + 8 * dim,
                "flops": rows * dim * 14}
    stored = n - (n // case["skip"] if case["skip"] else 0) if case["op"] == "append" else n
    moved = n * hq * dim * size * 2 + (n + stored) * hkv * dim * size
    if case["op"] == "append":
        moved = n * hq * dim * size * 2 + stored * hkv * dim * size * 4 + 4 * n
    return {"bytes": moved + angles + weights, "flops": rows * dim * (7 if case["norm"] else 3)}
