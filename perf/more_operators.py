"""Workloads of the 4-bit form of the paged cache: keys and values as OCP MX FP4
(E2M1 elements, one E8M0 scale for each 32 of a head).

``store``      a step's keys and values written into the cache: heads of q and k
               normalised and rotated, k and v quantised on the way, and the cache
               read back (what it holds is compared as the values it stands for)
``read``       cached rows read back as values, by slot
``attention``  attention of each sequence's new tokens over its 4-bit cache

A block of up to 32 elements of a head with the largest magnitude a has the
exponent e = the smallest in -124 .. 125 with a < 7 * 2^e (125 where none is), held
as the byte e + 127, and elements x held as the nearest of +-2^e {0, .5, 1, 1.5, 2, 3,
4, 6}, ties to the even code, larger ones as the largest.  A byte has the element 2i
in its low and 2i + 1 in its high four bits.  k is computed in 64 bits and rounded to
float32 before it is quantised, so that what is stored does not hang on the order
of sums.

``listed`` and ``draw`` give cases, ``prepare`` what a program holds before a
call, ``run`` one pass: in plain torch operations in 32 bits (64 for what is
quantised), or (``own``) through the library.  ``exact`` is the same result from the
definition in 64 bits, ``work`` the bytes and operations that a pass cannot do without.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 10000.0
BLOCK = 32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def _attention(name, mix, n_seqs, max_q, max_kv, hq, hkv, dim, page, window=0, causal=True,
               dtype="bf16"):
    return {"name": name, "op": "attention", "mix": mix, "n_seqs": n_seqs, "max_q": max_q,
            "max_kv": max_kv, "hq": hq, "hkv": hkv, "dim": dim, "page": page, "window": window,
            "causal": causal, "dtype": dtype}


def _store(name, tokens, hq, hkv, dim, rot, page, norm=True, adjacent=False, skip=0, dtype="bf16"):
    return {"name": name, "op": "store", "tokens": tokens, "hq": hq, "hkv": hkv, "dim": dim,
            "rot": rot, "page": page, "norm": norm, "adjacent": adjacent, "skip": skip,
            "dtype": dtype}


def _read(name, tokens, hkv, dim, page, skip=0, dtype="bf16"):
    return {"name": name, "op": "read", "tokens": tokens, "hkv": hkv, "dim": dim, "page": page,
            "skip": skip, "dtype": dtype}


def listed():
    return [
        # one user, one token: latency of a short context
        _attention("attention_decode_one", 1, 1, 1, 257, 16, 4, 128, 16),
        # a decode batch of 32 (width 4096) with contexts of all lengths
        _attention("attention_decode_batch", 2, 32, 1, 4096, 32, 8, 128, 16),
        # a few users with very long contexts, what a 4-bit cache is for
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
        _store("store_decode", 32, 32, 8, 128, 128, 16),
        # a prompt of 16384 tokens, some of them padding that is not stored
        _store("store_prompt", 16384, 32, 8, 128, 128, 64, skip=37),
        # a ragged float32 step: heads rotated in part, pairs side by side, a last block of 16
        _store("store_f32", 1001, 16, 4, 80, 40, 24, adjacent=True, dtype="f32"),
        # a long prefix moved out of the cache
        _read("read_prefix", 16384, 8, 128, 64),
        # a few rows of a small step, padding among them
        _read("read_few", 77, 4, 96, 24, skip=5, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    while True:
        case = _draw(rng)
        cost = work(case)
        # float32 products run at a sixteenth of the bfloat16 rate
        flops = cost["flops"] * (16 if case["dtype"] == "f32" else 1)
        scores = case["n_seqs"] * case["hq"] * case["max_q"] * case["max_kv"] \
            if case["op"] == "attention" else 0
        if cost["bytes"] < 4e8 and flops < 2e12 and scores < 5e9:
            return case


def _draw(rng):
    op = rng.choice(["attention"] * 5 + ["store"] * 3 + ["read"] * 2)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    hq, hkv = rng.choice([(32, 8), (16, 16), (16, 4), (8, 1), (28, 4), (40, 8), (5, 5)])
    dim = rng.choice([64, 80, 128, 128, 128, 256])
    page = rng.choice([1, 16, 24, 64, 256])
    if op != "attention":
        tokens = _log(rng, 1, 16384 * 32 * 128 // (hq * dim) if dtype == "bf16" else 4000)
        tokens, skip = min(tokens, 16384), rng.choice([0, 5, 37])
        if op == "read":
            return _read(None, tokens, hkv, dim, page, skip, dtype)
        return _store(None, tokens, hq, hkv, dim, rng.choice([dim, dim, dim // 2]), page,
                      rng.random() < 0.7, rng.random() < 0.3, skip, dtype)
    kind = rng.choice(["decode", "decode", "few", "chunk", "prompt"])
    mix, window = rng.randrange(1 << 30), rng.choice([0, 0, 0, _log(rng, 16, 4096)])
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


# ------------------------------------------------------- the format, plain form
def _blocks(dim):
    return -(-dim // BLOCK)


def _power(e):
    """2^e in float32, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """Codes [..., dim / 2] and scale bytes [..., blocks] of float32 x [..., dim]."""
    dim = x.shape[-1]
    y = torch.nn.functional.pad(x, (0, _blocks(dim) * BLOCK - dim)).unflatten(-1, (-1, BLOCK))
    top = y.abs().amax(-1)
    fine = torch.isfinite(top)
    part, power = torch.frexp(top)
    e = torch.where(fine & (top > 0), power - 3 + (part >= 0.875).int(), -124).clamp_(-124, 125)
    z = torch.where(fine[..., None], y * _power(-e)[..., None], 0.0)
    m = z.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0) + torch.signbit(z).to(torch.uint8) * 8)
    code = code.flatten(-2)[..., :dim]
    return code[..., 0::2] + code[..., 1::2] * 16, torch.where(fine, e + 127, 255).to(torch.uint8)


def _decode(codes, scales):
    """float32 values of codes [..., dim / 2] and their scale bytes."""
    both = torch.tensor(GRID + tuple(-g for g in GRID), device=codes.device)
    pairs = torch.stack([both.repeat(16), both.repeat_interleave(16)], 1)  # of every byte
    factor = torch.where(scales > 252, math.nan, _power(scales.int() - 127))
    factor = factor.repeat_interleave(BLOCK // 2, -1)[..., :codes.shape[-1], None]
    return (pairs[codes.int()] * factor).flatten(-2)


# ------------------------------------------------------------------ the inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _cache(gen, case, n_pages):
    """K and V as codes and scales: [page, token, head, ...] views of memory that has a
    page's tokens of one head side by side."""
    s = {}
    for n in "kv":
        x = _normal(gen, (n_pages, case["hkv"], case["page"], case["dim"]), _dtype(case))
        codes, scales = _encode(x.float())
        s[n + "_codes"], s[n + "_scales"] = codes.transpose(1, 2), scales.transpose(1, 2)
    if own:
        from activation_sparse_feed_amd import sffn
        s["cache"] = sffn.Mx4Cache(n_pages, case["page"], case["hkv"], case["dim"],
                                   k_codes=s["k_codes"], k_scales=s["k_scales"],
                                   v_codes=s["v_codes"], v_scales=s["v_scales"])
    return s


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
    s = {"case": case, **_cache(gen, case, n_pages),
         "q": _normal(gen, (tokens, case["hq"], dim), dt),
         "q_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
         "block_table": table}
    if own:
        from activation_sparse_feed_amd import sffn
        s["batch"] = sffn.make_paged_batch(
            tokens, len(kv_len), case["hq"], case["hkv"], dim, dt, page, n_pages, max(pages),
            max(q_len), max(kv_len), causal=case["causal"], window=case["window"])
        s["workspace"] = sffn.alloc_paged_mx4_workspace(s["batch"])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((tokens, case["hq"]), dtype=torch.float32, device="cuda")
    return s


def _slots(case, gen):
    """Rows of a cache of a few more pages, one for each token, -1 for padding."""
    n, page = case["tokens"], case["page"]
    n_pages = -(-n // page) + 5
    slots = torch.randperm(n_pages, generator=gen, device="cuda")[:, None] * page
    slots = (slots + torch.arange(page, device="cuda")[None, :]).reshape(-1)[:n].to(torch.int32)
    if case["skip"]:
        slots[case["skip"] - 1::case["skip"]] = -1
    return n_pages, slots


def _prepare_store(case, gen):
    n, hq, hkv, dim, dt = case["tokens"], case["hq"], case["hkv"], case["dim"], _dtype(case)
    # the projection's output: q, k and v side by side in one row of each token
    qkv = _normal(gen, (n, hq + 2 * hkv, dim), dt)
    max_pos = max(2 * n, 4096)
    n_pages, slots = _slots(case, gen)
    s = {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
         "q_weight": None, "k_weight": None, "table": _table(max_pos, case["rot"]),
         "positions": torch.randint(0, max_pos, (n,), generator=gen, device="cuda").to(torch.int32),
         "slots": slots, **_cache(gen, case, n_pages),
         "rows": torch.arange(n_pages * case["page"], dtype=torch.int32, device="cuda")}
    if case["norm"]:
        s["q_weight"] = (1 + _normal(gen, (dim,), torch.float32, 0.2)).to(dt)
        s["k_weight"] = (1 + _normal(gen, (dim,), torch.float32, 0.2)).to(dt)
    if own:
        from activation_sparse_feed_amd import sffn
        s["heads"] = sffn.make_heads(n, hq, hkv, dim, dt, rot_dim=case["rot"], max_pos=max_pos,
                                     norm=case["norm"], eps=EPS, adjacent=case["adjacent"])
        s["q_out"] = torch.empty((n, hq, dim), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((s["rows"].numel(), hkv, dim), dtype=dt, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    return s


def _prepare_read(case, gen):
    n_pages, slots = _slots(case, gen)
    # scattered, as a prefix of several sequences is; what a row without a slot holds stays
    slots = slots[torch.randperm(case["tokens"], generator=gen, device="cuda")].contiguous()
    shape = (case["tokens"], case["hkv"], case["dim"])
    return {"case": case, "slots": slots, **_cache(gen, case, n_pages),
            "k_out": _normal(gen, shape, _dtype(case)), "v_out": _normal(gen, shape, _dtype(case))}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"attention": _prepare_attention, "store": _prepare_store,
            "read": _prepare_read}[case["op"]](case, gen)


# ------------------------------------------------- one pass through the library
def _run_own(s):
    from activation_sparse_feed_amd import sffn
    op = s["case"]["op"]
    if op == "attention":
        sffn.paged_attn_mx4_fwd(s["batch"], s["q"], s["cache"], s["q_start"], s["kv_len"],
                                s["block_table"], s["out"], s["workspace"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "store":
        sffn.paged_kv_append_mx4(s["heads"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"],
                                 s["table"], s["positions"], s["slots"], s["q_out"], s["cache"])
        sffn.paged_kv_read_mx4(s["cache"], s["rows"], s["k_out"], s["v_out"])
        return s["q_out"], s["k_out"], s["v_out"]
    sffn.paged_kv_read_mx4(s["cache"], s["slots"], s["k_out"], s["v_out"])
    return s["k_out"], s["v_out"]


# ---------------------------------------------------------------- the plain form
def _plain_attention(s):
    """All sequences side by side, padded to the longest; float32."""
    case, dt = s["case"], s["q"].dtype
    hq, hkv, dim, page = case["hq"], case["hkv"], case["dim"], case["page"]
    g, ns = hq // hkv, case["n_seqs"]
    mq, mk = case["max_q"], case["max_kv"]
    j = torch.arange(mk, device="cuda")
    at = s["block_table"][:, j // page].long(), j % page                      # [ns, mk]
    k = _decode(s["k_codes"][at], s["k_scales"][at]).permute(0, 2, 3, 1).contiguous()
    i = torch.arange(mq, device="cuda")
    begin, n_new = s["q_start"][:-1, None], s["q_start"].diff()[:, None]
    row = (begin + i).clamp_(max=s["q"].shape[0] - 1)                         # [ns, mq]
    q = s["q"][row].float().view(ns, mq, hkv, g, dim).permute(0, 2, 1, 3, 4)
    p = torch.matmul(q.reshape(ns, hkv, mq * g, dim), k).mul_(1.0 / math.sqrt(dim))
    del k
    pos = (s["kv_len"][:, None] - n_new + i)[:, :, None]
    hide = j >= s["kv_len"][:, None, None]
    if case["causal"]:
        hide = hide | (j > pos)
    if case["window"]:
        hide = hide | (j <= pos - case["window"])
    p = p.view(ns, hkv, mq, g, mk)
    p.masked_fill_(hide[:, None, :, None, :], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = _decode(s["v_codes"][at], s["v_scales"][at]).permute(0, 2, 1, 3).contiguous()
    o = torch.matmul(p.view(ns, hkv, mq * g, mk), v).view(ns, hkv, mq, g, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(ns, mq, hq, dim)
    new = i < n_new
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    out[row[new]] = o[new].to(dt)
    lse[row[new]] = (top + total.log()).permute(0, 2, 1, 3, 4).reshape(ns, mq, hq)[new]
    return out, lse


def _pairs(x, rot, adjacent):
    """The two members of every rotated pair, and what is not rotated."""
    if adjacent:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _rotated(s, x, weight):
    case = s["case"]
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
    rot = case["rot"]
    c, z = s["table"].to(x.dtype)[s["positions"].long()][:, None, :].split(rot // 2, -1)
    a, b, rest = _pairs(x, rot, case["adjacent"])
    a, b = a * c - b * z, b * c + a * z
    both = torch.stack([a, b], -1).flatten(-2) if case["adjacent"] else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _plain_store(s):
    dt, page = s["q"].dtype, s["case"]["page"]
    q = _rotated(s, s["q"].float(), s["q_weight"]).to(dt)
    keep = s["slots"] >= 0
    slots = s["slots"][keep].long()
    at = slots // page, slots % page
    k = _rotated(s, s["k"].double(), s["k_weight"]).float()
    s["k_codes"][at], s["k_scales"][at] = _encode(k[keep])
    s["v_codes"][at], s["v_scales"][at] = _encode(s["v"][keep].float())
    return q, *(_decode(s[n + "_codes"], s[n + "_scales"]).flatten(0, 1).to(dt) for n in "kv")


def _plain_read(s):
    keep, page = s["slots"] >= 0, s["case"]["page"]
    slots = s["slots"][keep].long()
    at = slots // page, slots % page
    s["k_out"][keep] = _decode(s["k_codes"][at], s["k_scales"][at]).to(s["k_out"].dtype)
    s["v_out"][keep] = _decode(s["v_codes"][at], s["v_scales"][at]).to(s["v_out"].dtype)
    return s["k_out"], s["v_out"]


def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "store": _plain_store,
            "read": _plain_read}[state["case"]["op"]](state)


# ---------------------------------------------------- the definition in 64 bits
def _exact_values(codes, scales):
    """What codes and scale bytes stand for."""
    dim = 2 * codes.shape[-1]
    at = torch.arange(dim, device="cuda")
    code = (codes[..., at // 2].int() >> (4 * (at % 2)).int()) & 15
    m = code & 7
    # E2M1: two exponent bits with bias 1, one of the fraction
    x = torch.where(m < 2, m * 0.5, (2 + (m & 1)) * 0.5 * torch.exp2(((m >> 1) - 1).double()))
    x = torch.where(code >= 8, -x, x).double() * torch.exp2(scales[..., at // BLOCK].double() - 127)
    return torch.where(scales[..., at // BLOCK] >= 253, math.nan, x)


def _exact_quantised(x):
    """The values that stand for x (64 bits) in the cache."""
    x = x.float().double()
    res = torch.empty_like(x)
    for b in range(0, x.shape[-1], BLOCK):
        part = x[..., b:b + BLOCK]
        top = part.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 3
        for _ in range(3):
            e = torch.where(top >= 7 * torch.exp2(e), e + 1, e)
        scale = torch.exp2(e.clamp(-124, 125))
        m = part.abs() / scale
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
        m = (torch.round(m / step) * step).clamp(max=6.0)  # half way: to the even multiple
        res[..., b:b + BLOCK] = torch.where(torch.isfinite(top), torch.sign(part) * m * scale, math.nan)
    return res


def _exact_attention(s, q_len, kv_len):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for i, (nq, nkv) in enumerate(zip(q_len, kv_len)):
        j = torch.arange(nkv, device="cuda")
        page, off = s["block_table"][i].long()[j // case["page"]], j % case["page"]
        pos = torch.arange(nq, device="cuda")[:, None] + (nkv - nq)
        seen = torch.ones((nq, nkv), dtype=torch.bool, device="cuda")
        if case["causal"]:
            seen &= j[None, :] <= pos
        if case["window"]:
            seen &= pos - j[None, :] < case["window"]
        for h in range(hkv):
            k = _exact_values(s["k_codes"][page, off, h], s["k_scales"][page, off, h])
            v = _exact_values(s["v_codes"][page, off, h], s["v_scales"][page, off, h])
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
        x = x / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / dim + EPS) * weight.double()
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
        if len(q_len) * case["hq"] > 6000 or pairs * case["dim"] > 1.5e12:
            return None
        return _exact_attention(prepare(case, seed), q_len, kv_len)
    s = prepare(case, seed)
    held = {n: _exact_values(s[n + "_codes"], s[n + "_scales"]).flatten(0, 1) for n in "kv"}
    t = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][t].long()
    if case["op"] == "read":
        res = [s["k_out"].double(), s["v_out"].double()]
        res[0][t], res[1][t] = held["k"][slot], held["v"][slot]
        return res
    held["k"][slot] = _exact_quantised(_exact_rotated(s, s["k"].double(), s["k_weight"]))[t]
    held["v"][slot] = _exact_quantised(s["v"].double())[t]
    return _exact_rotated(s, s["q"].double(), s["q_weight"]), held["k"], held["v"]


# -------------------------------------------- what a pass cannot do without
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    hkv, dim, page = case["hkv"], case["dim"], case["page"]
    held = hkv * 2 * (dim // 2 + _blocks(dim))  # bytes of a token's keys and values
    if case["op"] == "attention":
        q_len, kv_len = _lengths(case)
        pairs = keys = 0
        for nq, nkv in zip(q_len, kv_len):
            keys += min(nkv, nq + case["window"] - 1) if case["window"] else nkv
            for pos in range(nkv - nq, nkv):
                end = pos + 1 if case["causal"] else nkv
                pairs += end - max(0, pos - case["window"] + 1) if case["window"] else end
        tokens, hq = sum(q_len), case["hq"]
        table = sum(-(-n // page) for n in kv_len) * 4 + 8 * len(kv_len) + 4
        return {"bytes": 2 * tokens * hq * dim * size + 4 * tokens * hq + keys * held + table,
                "flops": 4 * pairs * hq * dim}
    n = case["tokens"]
    stored = n - (n // case["skip"] if case["skip"] else 0)
    if case["op"] == "read":
        return {"bytes": stored * (held + 2 * hkv * dim * size) + 4 * n,
                "flops": 2 * stored * hkv * dim}
    hq, rows = case["hq"], (-(-n // page) + 5) * page
    angles = 4 * n + min(n, max(2 * n, 4096)) * case["rot"] * 4
    weights = 2 * dim * size if case["norm"] else 0
    # q, k and v in, q out, the rows stored; then all rows read back
    moved = 2 * n * hq * dim * size + stored * (2 * hkv * dim * size + held) + 4 * n
    moved += rows * (held + 2 * hkv * dim * size + 4)
    return {"bytes": moved + angles + weights,
            "flops": n * (hq + hkv) * dim * (7 if case["norm"] else 3) + (stored + rows) * 4 * hkv * dim}
