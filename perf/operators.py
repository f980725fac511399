"""Measured cases of the 8-bit document cache and of the norms around a decoder block.

The operators are ``kalm_cache_write`` (bf16 rows quantised into pages of a document cache),
``kalm_cache_read`` (pages back to packed bf16 rows), ``kalm_merged_attention_cache`` (the decoder's merged
self + cross attention reading its cross K/V from such pages) and ``kalm_rms_norm`` / ``kalm_norm_residual``
(the norm before a block; the norm after it with the gate, the residual and the next block's norm).

The cache holds e4m3 codes and, for each 32 consecutive columns of a row, one power-of-two scale 2^e as the
byte e + 127: e is the least integer with max|v| <= 448 * 2^e, at least -120; a code is v * 2^-e rounded to
nearest even (at most 240 where e is 120, so that every stored value is a bf16 number).

With ``own`` false, ``run`` computes the operators by elementary torch operations in 32 bits; with ``own`` true
it makes the calls that a user of the package makes.
"""
import math
import random

import torch

own = False

HEAD_DIM = 256
GROUP = 32  # columns that share a scale


# --------------------------------------------------------------------------------------------- sizes of a case
def doc_rows(case):
    """Cached rows of each document: its encoder tokens, by the case's law, in chunks."""
    rng = random.Random(case["len_seed"])
    lo, hi = case["len_lo"], case["len_hi"]
    if case["law"] == "lognormal":
        tokens = [min(hi, max(lo, round(rng.lognormvariate(math.log(200.0), 0.6)))) for _ in range(case["n_docs"])]
    else:
        tokens = [rng.randint(lo, hi) for _ in range(case["n_docs"])]
    return [-(-t // case["chunk"]) for t in tokens]


def first_rows(case):
    """Rows that each document holds already, where the new ones are appended."""
    rng = random.Random(case["len_seed"] + 1)
    return [rng.randint(0, case["held"]) for _ in range(case["n_docs"])]


def query_rows(case):
    """Decoder rows of each document."""
    if not case["ragged"]:
        return [case["lq"]] * case["n_docs"]
    rng = random.Random(case["len_seed"] + 2)
    return [rng.randint(1, case["lq"]) for _ in range(case["n_docs"])]


def listed():
    return [
        # one more pooled vector of one document joins the cache: the smallest call
        dict(name="write one row", op="write", n_docs=1, law="uniform", len_lo=4, len_hi=4, chunk=4, len_seed=1, held=40,
             width=640, page_rows=64),
        # the pooled vectors of a sweep point's documents, as they leave the pooling
        dict(name="write pooled 1024 docs", op="write", n_docs=1024, law="lognormal", len_lo=1, len_hi=1024, chunk=4,
             len_seed=2, held=0, width=640, page_rows=16),
        # every layer's cross K and V of the Nano shape's documents
        dict(name="write cross kv nano", op="write", n_docs=100, law="uniform", len_lo=64, len_hi=1024, chunk=4, len_seed=3,
             held=0, width=9216, page_rows=64),
        # a handful of cached documents read back for a short query
        dict(name="read pooled 4 docs", op="read", n_docs=4, law="uniform", len_lo=1, len_hi=64, chunk=4, len_seed=4, held=3,
             width=640, page_rows=16),
        # the candidates of one query read back, the widest pooled vectors
        dict(name="read pooled 1024 docs", op="read", n_docs=1024, law="lognormal", len_lo=16, len_hi=1024, chunk=4,
             len_seed=5, held=0, width=2560, page_rows=64),
        # a few documents, a short query
        dict(name="attention 4 docs", op="attention", n_docs=4, law="uniform", len_lo=1, len_hi=64, chunk=4, len_seed=6,
             lq=32, ragged=False, shared=False, n_q=4, n_kv=1, layers=1, page_rows=16, lse=True),
        # one decoder position per document: a step that adds a single token
        dict(name="attention one position", op="attention", n_docs=100, law="uniform", len_lo=64, len_hi=1024, chunk=4,
             len_seed=7, lq=1, ragged=False, shared=False, n_q=4, n_kv=1, layers=18, page_rows=64, lse=False),
        # one layer of the Nano shape
        dict(name="attention nano", op="attention", n_docs=100, law="uniform", len_lo=64, len_hi=1024, chunk=4, len_seed=8,
             lq=128, ragged=False, shared=False, n_q=4, n_kv=1, layers=18, page_rows=64, lse=False),
        # one layer of the Large shape
        dict(name="attention large", op="attention", n_docs=100, law="lognormal", len_lo=16, len_hi=1024, chunk=4,
             len_seed=9, lq=256, ragged=False, shared=False, n_q=8, n_kv=4, layers=4, page_rows=32, lse=False),
        # the norm before the first block of one decoder row
        dict(name="norm one row", op="norm", n_docs=1, law="uniform", len_lo=1, len_hi=1, chunk=1, len_seed=10, width=640,
             post=False, gate="none", pre=True),
        # between two blocks of the Nano shape, one gate for all documents
        dict(name="norm nano", op="norm", n_docs=100, law="uniform", len_lo=128, len_hi=128, chunk=1, len_seed=11, width=640,
             post=True, gate="row", pre=True),
        # between two blocks of the Large shape, a gate for each document, documents of several lengths
        dict(name="norm large ragged", op="norm", n_docs=100, law="uniform", len_lo=1, len_hi=511, chunk=1, len_seed=12,
             width=2560, post=True, gate="doc", pre=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "attention", "attention", "norm"])
    case = dict(op=op, n_docs=log(1, 1024), law=rng.choice(["uniform", "lognormal"]), len_lo=rng.randint(1, 64),
                len_hi=log(64, 1024), chunk=rng.choice([1, 2, 4, 4, 8]), len_seed=rng.randrange(1 << 30))
    if op in ("write", "read"):
        case |= dict(held=log(1, 256) - 1, width=GROUP * log(1, 288), page_rows=1 << rng.randint(3, 8))
    elif op == "attention":
        n_kv = rng.choice([1, 1, 2, 4])
        case |= dict(lq=log(1, 512), ragged=rng.random() < 0.5, shared=rng.random() < 0.25, n_q=n_kv * rng.choice([1, 2, 4, 8]),
                     n_kv=n_kv, layers=rng.randint(1, 4), page_rows=1 << rng.randint(3, 8), lse=rng.random() < 0.3)
    else:
        post = rng.random() < 0.75
        case |= dict(width=8 * log(1, 1024), post=post, gate=rng.choice(["none", "row", "doc"]) if post else "none",
                     pre=(not post) or rng.random() < 0.75)
    most = {m: max(work(c)[m] for c in listed() if c["op"] == op) for m in ("bytes", "flops")}
    while any(work(case)[m] > most[m] for m in most) or padded(case) > 100 * 256:
        case["n_docs"] = case["n_docs"] * 3 // 4
    return case


def padded(case):
    """Rows of the plain attention's padded score matrices, for a cap on its memory."""
    return case["n_docs"] * case["lq"] * case["n_q"] // 8 if case["op"] == "attention" else 0


def work(case):
    rows = doc_rows(case)
    total = sum(rows)
    if case["op"] in ("write", "read"):
        return {"bytes": total * case["width"] * (2 + 1 + 1 / GROUP) + 8 * case["n_docs"], "flops": 0.0}
    if case["op"] == "attention":
        lq, d = query_rows(case), HEAD_DIM
        n_q, n_kv = case["n_q"], case["n_kv"]
        read = (max(lq) if case["shared"] else sum(lq)) * (n_q + 2 * n_kv) * d * 2
        cached = total * 2 * n_kv * (d + d // GROUP)
        pairs = sum(a * (a + 1) // 2 + a * b for a, b in zip(lq, rows))
        return {"bytes": float(read + cached + sum(lq) * n_q * d * 2), "flops": 4.0 * d * n_q * pairs}
    tensors = (3 if case["post"] else 1) + (1 if case["pre"] else 0)
    return {"bytes": float(total * case["width"] * 2 * tensors), "flops": 0.0}


# --------------------------------------------------------------------------------------------- inputs
def offsets(counts, device):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return torch.tensor(off, dtype=torch.int64, device=device)


def pages(counts, page_rows, gen, device):
    """A page table for documents of `counts` rows over shuffled pages, and the number of pages."""
    need = [-(-c // page_rows) for c in counts]
    n_pages = sum(need) + 3  # a few belong to other documents
    perm = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32)
    table = torch.full((len(counts), max(max(need), 1)), -1, dtype=torch.int32, device=device)
    start = offsets(need, device)
    used = torch.arange(table.shape[1], device=device)[None, :] < (start[1:] - start[:-1])[:, None]
    table[used] = perm[: sum(need)]
    return table, n_pages


def cache_content(rows, width, gen, device, spread):
    """Codes and scales of a filled cache: normal values with a spread of magnitudes per row and column."""
    codes = torch.empty(rows, width, dtype=torch.uint8, device=device)
    scales = torch.empty(rows, width // GROUP, dtype=torch.uint8, device=device)
    step = max(1, (1 << 26) // width)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        v = torch.randn(n, width, generator=gen, device=device) * spread
        codes[r:r + n], scales[r:r + n] = quantise(v.to(torch.bfloat16))
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std + mean).to(torch.bfloat16)

    op, rows = case["op"], doc_rows(case)
    s = {"case": case, "off": offsets(rows, dev)}
    total = sum(rows)
    if op in ("write", "read"):
        first = first_rows(case)
        s["first"] = torch.tensor(first, dtype=torch.int32, device=dev) if case["held"] else None
        s["table"], n_pages = pages([a + b for a, b in zip(rows, first)], case["page_rows"], gen, dev)
        n = n_pages * case["page_rows"]
        if op == "write":
            # encoder-like rows: each column has a size of its own, a few are far larger than the rest
            size = torch.exp(0.5 * torch.randn(case["width"], generator=gen, device=dev))
            s["src"] = (torch.randn(total, case["width"], generator=gen, device=dev) * size).to(torch.bfloat16)
            s["codes"] = torch.zeros(n, case["width"], dtype=torch.uint8, device=dev)
            s["scales"] = torch.zeros(n, case["width"] // GROUP, dtype=torch.uint8, device=dev)
        else:
            s["codes"], s["scales"] = cache_content(n, case["width"], gen, dev, 1.0)
            s["dst"] = torch.empty(total, case["width"], dtype=torch.bfloat16, device=dev)
    elif op == "attention":
        d, n_q, n_kv = HEAD_DIM, case["n_q"], case["n_kv"]
        lq = query_rows(case)
        s["q_off"] = offsets(lq, dev)
        n_in = max(lq) if case["shared"] else sum(lq)
        s["qkv"] = normal(n_in, (n_q + 2 * n_kv) * d, std=0.7)
        s["in_off"] = torch.zeros(case["n_docs"], dtype=torch.int64, device=dev) if case["shared"] else None
        s["table"], n_pages = pages(rows, case["page_rows"], gen, dev)
        s["layer"] = seed % case["layers"]
        s["codes"], s["scales"] = cache_content(n_pages * case["page_rows"], case["layers"] * 2 * n_kv * d, gen, dev, 0.7)
        s["out"] = torch.empty(sum(lq), n_q * d, dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty(sum(lq), n_q, dtype=torch.float32, device=dev) if case["lse"] else None
        s["max_q"], s["order"] = max(lq), None
        if own:  # the plan that a program keeps for a query's layers
            import encoder_decoder_document_b200 as kalm
            items = kalm.kalm_attention_items(case["n_docs"], s["max_q"], n_q, n_kv)
            s["order"] = torch.empty(items, dtype=torch.int32, device=dev)
            kalm.kalm_attention_schedule(s["q_off"], s["off"], s["max_q"], n_q, n_kv, s["order"])
    else:
        w = case["width"]
        s["x"] = normal(total, w, std=2.0)
        s["w_pre"] = normal(w, std=0.2) if case["pre"] else None
        s["h"] = torch.empty(total, w, dtype=torch.bfloat16, device=dev) if case["pre"] else None
        if case["post"]:
            s["y"] = normal(total, w, std=0.3)
            s["w_post"] = normal(w, std=0.2)
            s["gate"] = {"none": lambda: None, "row": lambda: normal(w, std=0.3, mean=1.0),
                         "doc": lambda: normal(case["n_docs"], w, std=0.3, mean=1.0)}[case["gate"]]()
            s["x_out"] = torch.empty(total, w, dtype=torch.bfloat16, device=dev)
    return s


EPS, RESIDUAL_SCALE, WEIGHT_OFFSET = 1e-6, 0.9, 1.0


# --------------------------------------------------------------------------------------------- plain forms
def power_of_two(e):
    """2^e in 32 bits, from its exponent field."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def quantise(v):
    """Codes and scale bytes of rows of bf16 values."""
    g = v.float().unflatten(-1, (-1, GROUP))
    fine = torch.isfinite(g)
    top = torch.where(fine, g.abs(), 0.0).amax(-1, keepdim=True)
    m, x = torch.frexp(top)  # top = m 2^x, 448 = 0.875 * 2^9
    e = torch.where(top > 0, x - 9 + (m > 0.875).to(x.dtype), -120).clamp(min=-120)
    lim = torch.where(e >= 120, 240.0, 448.0)
    t = (g * power_of_two(-e)).clamp(min=-lim, max=lim)
    t = torch.where(fine, t, float("nan")).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).flatten(-2), (e + 127).squeeze(-1).to(torch.uint8)


def values(codes, scales):
    """The numbers that codes and scale bytes stand for."""
    f = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, GROUP))
    return (f * power_of_two(scales.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def cache_index(off, first, table, page_rows, total):
    """Cache row of each packed row."""
    r = torch.arange(total, device=off.device)
    d = torch.searchsorted(off, r, right=True) - 1
    at = r - off[d] + (first[d].long() if first is not None else 0)
    return table[d, at // page_rows].long() * page_rows + at % page_rows


def plain_attention(s):
    case, d = s["case"], HEAD_DIM
    n_docs, n_q, n_kv, lq = case["n_docs"], case["n_q"], case["n_kv"], s["max_q"]
    dev = s["qkv"].device
    g = n_q // n_kv
    q_len, c_len = s["q_off"][1:] - s["q_off"][:-1], s["off"][1:] - s["off"][:-1]
    nc = s["table"].shape[1] * case["page_rows"]
    # the documents' rows, padded
    pos, col = torch.arange(lq, device=dev), torch.arange(nc, device=dev)
    start = s["in_off"] if s["in_off"] is not None else s["q_off"][:-1]
    row = torch.where(pos < q_len[:, None], start[:, None] + pos, 0)
    x = s["qkv"][row].float()
    q = x[..., : n_q * d].reshape(n_docs, lq, n_kv, g, d).permute(0, 2, 3, 1, 4).reshape(n_docs, n_kv, g * lq, d)
    ks = x[..., n_q * d:(n_q + n_kv) * d].reshape(n_docs, lq, n_kv, d).transpose(1, 2)
    vs = x[..., (n_q + n_kv) * d:].reshape(n_docs, lq, n_kv, d).transpose(1, 2)
    at = s["table"].clamp(min=0).long()[:, col // case["page_rows"]] * case["page_rows"] + col % case["page_rows"]
    kv = slice(s["layer"] * 2 * n_kv * d, (s["layer"] + 1) * 2 * n_kv * d)
    sc = slice(kv.start // GROUP, kv.stop // GROUP)
    c = values(s["codes"][:, kv][at], s["scales"][:, sc][at])
    kc = c[..., : n_kv * d].reshape(n_docs, nc, n_kv, d).transpose(1, 2)
    vc = c[..., n_kv * d:].reshape(n_docs, nc, n_kv, d).transpose(1, 2)
    # one softmax over the causal self keys and the document's cross keys
    a = torch.matmul(q, torch.cat([ks, kc], 2).transpose(2, 3)) * d ** -0.5
    seen = torch.cat([(pos[None, :] <= pos[:, None]).expand(n_docs, lq, lq),
                      (col[None, :] < c_len[:, None])[:, None, :].expand(n_docs, lq, nc)], 2)
    a = a.view(n_docs, n_kv, g, lq, lq + nc).masked_fill_(~seen[:, None, None], float("-inf"))
    top = a.amax(-1, keepdim=True)
    p = a.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    v = torch.cat([vs, torch.where((col < c_len[:, None])[:, None, :, None], vc, 0.0)], 2)
    o = torch.matmul(p.view(n_docs, n_kv, g * lq, lq + nc), v).view(n_docs, n_kv, g, lq, d) / z
    keep = pos < q_len[:, None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[keep].reshape(-1, n_q * d))
    if s["lse"] is not None:
        s["lse"].copy_((top + z.log()).squeeze(-1).permute(0, 3, 1, 2)[keep].reshape(-1, n_q))


def plain_norm(v, w):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * (w.float() + WEIGHT_OFFSET)


def run(s):
    """One call of the case's operator."""
    case = s["case"]
    op = case["op"]
    if own:
        import encoder_decoder_document_b200 as kalm
    if op == "write":
        if own:
            kalm.kalm_cache_write(s["src"], s["off"], s["table"], case["page_rows"], s["codes"], s["scales"], first_row=s["first"])
        else:
            at = cache_index(s["off"], s["first"], s["table"], case["page_rows"], s["src"].shape[0])
            s["codes"][at], s["scales"][at] = quantise(s["src"])
        # the codes as the numbers they are, the scales' exponents as whole numbers
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    if op == "read":
        if own:
            kalm.kalm_cache_read(s["codes"], s["scales"], s["off"], s["table"], case["page_rows"], s["dst"], first_row=s["first"])
        else:
            at = cache_index(s["off"], s["first"], s["table"], case["page_rows"], s["dst"].shape[0])
            s["dst"].copy_(values(s["codes"][at], s["scales"][at]))
        return s["dst"]
    if op == "attention":
        if own:
            d, n_q, n_kv = HEAD_DIM, case["n_q"], case["n_kv"]
            k, v = s["layer"] * 2 * n_kv * d, (s["layer"] * 2 + 1) * n_kv * d
            w = n_kv * d
            kalm.kalm_merged_attention_cache(
                s["qkv"][:, : n_q * d], s["qkv"][:, n_q * d:n_q * d + w], s["qkv"][:, n_q * d + w:],
                s["codes"][:, k:k + w], s["scales"][:, k // GROUP:(k + w) // GROUP],
                s["codes"][:, v:v + w], s["scales"][:, v // GROUP:(v + w) // GROUP], s["table"], case["page_rows"],
                s["q_off"], s["off"], s["max_q"], n_q, n_kv, s["out"], lse=s["lse"], in_off=s["in_off"], order=s["order"])
        else:
            plain_attention(s)
        return {"out": s["out"], "lse": s["lse"]}
    if not case["post"]:
        if own:
            kalm.kalm_rms_norm(s["x"], s["w_pre"], s["h"], eps=EPS, weight_offset=WEIGHT_OFFSET)
        else:
            s["h"].copy_(plain_norm(s["x"].float(), s["w_pre"]))
        return s["h"]
    if own:
        kalm.kalm_norm_residual(s["y"], s["x"], s["x_out"], h=s["h"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                                q_off=s["off"], residual_scale=RESIDUAL_SCALE, eps=EPS, weight_offset=WEIGHT_OFFSET)
    else:
        u = plain_norm(s["y"].float(), s["w_post"])
        if case["gate"] == "row":
            u = u * s["gate"].float()
        elif case["gate"] == "doc":
            r = torch.arange(u.shape[0], device=u.device)
            u = u * s["gate"][torch.searchsorted(s["off"], r, right=True) - 1].float()
        t = RESIDUAL_SCALE * s["x"].float() + u
        s["x_out"].copy_(t)
        if case["pre"]:
            s["h"].copy_(plain_norm(t, s["w_pre"]))
    return {"x": s["x_out"], "h": s["h"]}


# --------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    off = s["off"].tolist()

    def cache_rows(i):
        """Cache rows of document i's packed rows, one page at a time."""
        first = int(s["first"][i]) if s.get("first") is not None else 0
        j = torch.arange(first, first + off[i + 1] - off[i], device=s["table"].device)
        page = s["table"][i].long()[torch.div(j, case["page_rows"], rounding_mode="floor")]
        return page * case["page_rows"] + torch.remainder(j, case["page_rows"])

    def pow2(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    def number(codes, scales):
        """sign * mantissa * 2^exponent of e4m3 codes, times their scales."""
        c = codes.long()
        expo, frac = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(expo == 0, frac / 512.0, (1.0 + frac / 8.0) * pow2(expo - 7))
        mag = torch.where(c >= 128, -mag, mag)
        return mag * pow2(scales.long() - 127).repeat_interleave(GROUP, -1)

    if op == "write":
        codes = s["codes"].double()
        scales = s["scales"].double()
        for i in range(case["n_docs"]):
            v = s["src"][off[i]:off[i + 1]].double()
            w = v.reshape(v.shape[0], -1, GROUP)
            e = torch.ceil(torch.log2(w.abs().amax(-1) / 448.0) - 1e-12).clamp(min=-120.0)
            t = w / pow2(e)[..., None]
            grid = pow2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)) + 1e-12) - 3)  # e4m3's step at t
            at = cache_rows(i)
            codes[at] = (torch.round(t / grid) * grid).clamp(-448.0, 448.0).reshape(v.shape)
            scales[at] = e + 127.0
        return {"codes": codes, "scales": scales.long()}
    if op == "read":
        return torch.cat([number(s["codes"][cache_rows(i)], s["scales"][cache_rows(i)]) for i in range(case["n_docs"])])
    if op == "attention":
        d, n_q, n_kv = HEAD_DIM, case["n_q"], case["n_kv"]
        q_off = s["q_off"].tolist()
        out, lse = [], []
        for i in range(case["n_docs"]):
            lq = q_off[i + 1] - q_off[i]
            at = 0 if case["shared"] else q_off[i]
            x = s["qkv"][at:at + lq].double().view(lq, n_q + 2 * n_kv, d)
            rows = cache_rows(i)
            w = 2 * n_kv * d
            c = number(s["codes"][rows, s["layer"] * w:(s["layer"] + 1) * w],
                       s["scales"][rows, s["layer"] * w // GROUP:(s["layer"] + 1) * w // GROUP]).view(len(rows), 2, n_kv, d)
            heads, dens = [], []
            for h in range(n_q):
                g = h // (n_q // n_kv)
                own_part = x[:, h] @ x[:, n_q + g].T / math.sqrt(d)
                own_part = own_part + torch.full_like(own_part, float("-inf")).triu(1)
                logits = torch.cat([own_part, x[:, h] @ c[:, 0, g].T / math.sqrt(d)], 1)
                dens.append(torch.logsumexp(logits, 1))
                heads.append(torch.softmax(logits, 1) @ torch.cat([x[:, n_q + n_kv + g], c[:, 1, g]]))
            out.append(torch.stack(heads, 1).reshape(lq, n_q * d))
            lse.append(torch.stack(dens, 1))
        return {"out": torch.cat(out), "lse": torch.cat(lse) if case["lse"] else None}

    def unit(v):
        return v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS)

    x = s["x"].double()
    if not case["post"]:
        return unit(x) * (WEIGHT_OFFSET + s["w_pre"].double())
    u = unit(s["y"].double()) * (WEIGHT_OFFSET + s["w_post"].double())
    if case["gate"] != "none":
        gate = s["gate"].double()
        if case["gate"] == "doc":
            gate = torch.repeat_interleave(gate, s["off"][1:] - s["off"][:-1], 0)
        u = u * gate
    x = RESIDUAL_SCALE * x + u
    return {"x": x, "h": unit(x) * (WEIGHT_OFFSET + s["w_pre"].double()) if case["pre"] else None}
