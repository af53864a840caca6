"""Cases of the paged 8-bit cache's operators: append (with the position rotation), attend
and gather. ``run`` computes them in plain torch, or through the package when ``own``.

Cache layout: codes [n_pages][H][P][d] (e4m3), one power-of-two fp32 scale per (page, head);
token t of sequence b is row t % P of page table[b][t // P]; a value is code * scale.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
THETA = 5e5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest call: one generated token of one sequence, the small fp32 shape
        dict(name="append one token, f32 d64", kind="append", dtype="f32", heads=2, group=4, dim=64,
             page=16, batch=1, longest=300, new=1, ragged=False),
        # one decode step's keys and values of a batch, each sequence at its own length
        dict(name="append step, batch 8", kind="append", dtype="bf16", heads=8, group=4, dim=128,
             page=16, batch=8, longest=4100, new=1, ragged=False),
        # prompts of different lengths written in one call, behind what is cached already
        dict(name="append ragged prompts", kind="append", dtype="bf16", heads=8, group=4, dim=128,
             page=64, batch=6, longest=9000, new=7000, ragged=True),
        # the start of a generation: under a hundred tokens
        dict(name="attend short, f32 d64", kind="attend", dtype="f32", heads=2, group=4, dim=64,
             page=16, batch=1, longest=77, queries=1),
        # one sequence with a generated suffix of a few thousand tokens
        dict(name="attend one sequence 4K", kind="attend", dtype="bf16", heads=8, group=4, dim=128,
             page=16, batch=1, longest=4099, queries=1),
        # serving: a batch of many requests, every length from empty to some thousands
        dict(name="attend batch 28 ragged", kind="attend", dtype="bf16", heads=8, group=4, dim=128,
             page=32, batch=28, longest=9001, queries=1),
        # checking a few drafted tokens in one pass
        dict(name="attend 5 drafted tokens 16K", kind="attend", dtype="bf16", heads=8, group=4, dim=128,
             page=16, batch=4, longest=16500, queries=5),
        # the fp32 form with 64-wide heads, long and ragged
        dict(name="attend f32 d64 ragged 40K", kind="attend", dtype="f32", heads=4, group=8, dim=64,
             page=64, batch=12, longest=40001, queries=1),
        # the uncompressed alternative to the long prefix: batch 8 at 128K tokens
        dict(name="attend batch 8 128K", kind="attend", dtype="bf16", heads=8, group=4, dim=128,
             page=64, batch=8, longest=131072, queries=1),
        # a short block read back, one sequence ending inside it
        dict(name="gather 200 tokens f32 d64", kind="gather", dtype="f32", heads=2, group=4, dim=64,
             page=16, batch=2, longest=500, count=200),
        # the suffix block that is compressed next: 4K tokens of every sequence
        dict(name="gather 4K tokens batch 8", kind="gather", dtype="bf16", heads=8, group=4, dim=128,
             page=16, batch=8, longest=6000, count=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "gather"])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "f32"]), heads=rng.choice([1, 2, 4, 8]),
             group=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]))
    if kind == "append":
        c["ragged"] = rng.random() < 0.6
        c["new"] = _log(rng, 1, 6000)
        c["batch"] = _log(rng, 1, 32 if c["new"] < 600 else 6)
        c["longest"] = c["new"] + _log(rng, 1, 4000)
    elif kind == "attend":
        c["batch"] = _log(rng, 1, 32)
        c["longest"] = _log(rng, 5, 131072 if c["batch"] <= 4 else 20000)
        c["queries"] = rng.choice([1, 1, 1, rng.randint(2, 16)])
    else:
        c["batch"] = _log(rng, 1, 16)
        c["count"] = _log(rng, 8, 6000)
        c["longest"] = c["count"] + _log(rng, 1, 3000)
    return c


# ------------------------------------------------------------------------------- inputs
def _lens(case):
    """Lengths as plain numbers from the case alone: the first sequence has the longest, one of
    a batch of five or more is empty (not where tokens are appended), the others lie between."""
    n, top = case["batch"], case["longest"]
    out = [top - (i * 7919 * top // 16384) % max(1, (3 * top) // 4) for i in range(n)]
    if n >= 5 and case["kind"] != "append" and top < 100000:
        out[3] = 0
    if top >= 100000:
        out = [top - 13 * i for i in range(n)]
    return out


def _new(case, lens):
    if not case["ragged"]:
        return [min(case["new"], min(lens))] * len(lens)
    return [max(0, min(l, case["new"] - (i * 5 * case["new"]) // (4 * len(lens) + 1)))
            for i, l in enumerate(lens)]


def _starts(case):
    return [(b * 37) % max(1, case["longest"] - case["count"]) for b in range(case["batch"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    H, d, P, B = case["heads"], case["dim"], case["page"], case["batch"]
    lens = _lens(case)
    max_pages = max(1, max(-(-l // P) for l in lens)) + 1
    n_pages = sum(-(-l // P) for l in lens) + 3
    s = {"case": case}

    def pool():
        x = torch.empty(n_pages, H, P, d, dtype=torch.uint8, device=dev)
        for i in range(0, n_pages, 4096):
            y = torch.randn(x[i:i + 4096].shape, generator=g, device=dev, dtype=torch.float16)
            x[i:i + 4096] = (y * 96).clamp_(-448, 448).to(FP8).view(torch.uint8)
        e = torch.randint(-8, -5, (n_pages, H), generator=g, device=dev)
        return x, torch.exp2(e.float())

    s["k_code"], s["k_scale"] = pool()
    s["v_code"], s["v_scale"] = pool()
    # pages lie anywhere in the pool; what is behind a sequence's last page is never looked at
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, max_pages, dtype=torch.int32, device=dev)
    at = 0
    for b, l in enumerate(lens):
        k = -(-l // P)
        table[b, :k] = order[at:at + k]
        at += k
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["kind"] == "append":
        new = _new(case, lens)
        n = sum(new)
        s["k_new"] = torch.randn(n, H, d, generator=g, device=dev).to(dt)
        s["v_new"] = torch.randn(n, H, d, generator=g, device=dev).to(dt)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if case["ragged"] else None
        s["max_new"] = max(new)
        # the suffix begins behind a compressed prefix: its first position, by sequence
        s["base"] = torch.tensor([32768 + 4096 * b for b in range(B)], dtype=torch.int32, device=dev)
    elif case["kind"] == "attend":
        hq, nq = H * case["group"], case["queries"]
        s["q"] = torch.randn(B, nq, hq, d, generator=g, device=dev).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, nq, hq, dtype=torch.float32, device=dev)
    else:
        n = case["count"]
        # the block to compress begins at a page, or where the last one ended
        s["start"] = torch.tensor(_starts(case), dtype=torch.int32, device=dev)
        s["k_out"] = torch.empty(B, n, H, d, dtype=dt, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        from long_context_decode_02_b200 import lowram as L
        cfg = L.lowram_config(
            batch=B, n_tokens=16, n_kv_heads=H, n_q_heads=H * case["group"], head_dim=d, rank=16,
            chunk=1, mlp_hidden=128, top_k=1, n_res=0, act=L.ACT_SILU,
            dtype=L.DTYPE_BF16 if case["dtype"] == "bf16" else L.DTYPE_F32,
            decode_variant=L.DECODE_AUTO, res_format=L.RES_STORE, n_positions=0, reserved=0,
            rope_theta=THETA)
        s["ctx"] = L.Context(cfg, 0)
        s["pages"] = L.paged_cache(s["k_code"], s["v_code"], s["k_scale"], s["v_scale"], table,
                                   s["lens"])
        if case["kind"] == "attend":
            size = L.paged_workspace_size(cfg, B, case["queries"])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------- plain forms
def _scale_for(amax):
    """The smallest power of two 2^e, e >= -64, with amax <= 448 * 2^e = 0.875 * 2^(e + 9)."""
    m, x = torch.frexp(amax)
    e = torch.where(m > 0.875, x - 8, x - 9)
    e = torch.where(amax == 0, torch.full_like(e, -64), e).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), e)


def _rotate(x, pos, dim):
    """Rotate-half position rotation with angles and products in 64 bits."""
    i = torch.arange(dim // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None] * torch.pow(torch.tensor(THETA, dtype=torch.float64,
                                                         device=x.device), -2.0 * i / dim)
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x.double().chunk(2, dim=-1)
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1).float()


def _plain_append(s):
    case = s["case"]
    d, P, B = case["dim"], case["page"], case["batch"]
    lens, table = s["lens"].long(), s["table"].long()
    n = s["k_new"].shape[0]
    if s["cu"] is None:
        cu = torch.arange(B + 1, device=lens.device) * (n // B)
    else:
        cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    t = torch.arange(n, device=lens.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    first = lens - count
    idx = first[b] + t - cu[b]
    page, row = table[b, idx // P], idx % P
    # pages that held tokens of their sequence before this call
    part = (count > 0) & (first % P > 0)
    old_page = table[torch.arange(B, device=lens.device), (first // P).clamp(max=table.shape[1] - 1)]
    for name, x in (("k", _rotate(s["k_new"], s["base"].long()[b] + idx, d)), ("v", s["v_new"].float())):
        code, scale = s[name + "_code"], s[name + "_scale"]
        amax = torch.full_like(scale, -1.0).index_reduce_(0, page, x.abs().amax(dim=-1), "amax")
        fresh = _scale_for(amax.clamp(min=0))
        keep = torch.zeros(scale.shape[0], dtype=torch.bool, device=scale.device)
        keep.index_fill_(0, old_page[part], True)
        now = torch.where(keep[:, None], torch.maximum(fresh, scale), fresh)
        now = torch.where(amax >= 0, now, scale)
        # earlier rows of those pages, at the page's new scale
        p = old_page[part]
        before = torch.arange(P, device=lens.device)[None] < (first[part] % P)[:, None]
        ratio = (scale[p] / now[p])[:, :, None, None]
        again = (code[p].view(FP8).float() * ratio).to(FP8).view(torch.uint8)
        code[p] = torch.where(before[:, None, :, None], again, code[p])
        scale.copy_(now)
        code[page, :, row] = (x / now[page][:, :, None]).to(FP8).view(torch.uint8)
    return _pools(s)


def _pools(s):
    return {n: s[n].view(FP8) if n.endswith("code") else s[n]
            for n in ("k_code", "k_scale", "v_code", "v_scale")}


def _plain_attend(s):
    case = s["case"]
    G, P = case["group"], case["page"]
    q = s["q"].float()
    B, nq, hq, d = q.shape
    H = hq // G
    lens = s["lens"].long()
    used = s["table"].long()

    def values(name):   # [B][H][T][d]
        x = s[name + "_code"][used].view(FP8).float() * s[name + "_scale"][used][..., None, None]
        return x.transpose(1, 2).reshape(B, H, -1, d)

    q = q.view(B, nq, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, d)
    z = (q @ values("k").transpose(2, 3)) * (1.0 / math.sqrt(d))
    T = z.shape[-1]
    t = torch.arange(T, device=q.device)
    last = lens[:, None] - nq + torch.arange(nq, device=q.device)          # [B][nq]
    seen = (t[None, None] <= last[..., None])[:, None, :, None]            # [B][1][nq][1][T]
    z = z.view(B, H, nq, G, T).masked_fill(~seen, -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = e.sum(dim=-1, keepdim=True)
    out = (e.view(B, H, nq * G, T) @ values("v")).view(B, H, nq, G, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log()).squeeze(-1)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, nq, hq, d).to(s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, nq, hq)}


def _plain_gather(s):
    case = s["case"]
    P, B, n = case["page"], case["batch"], case["count"]
    idx = s["start"].long()[:, None] + torch.arange(n, device="cuda")      # [B][n]
    held = idx < s["lens"].long()[:, None]
    page = s["table"].long().gather(1, (idx // P).clamp(max=s["table"].shape[1] - 1))
    res = {}
    for name in ("k", "v"):
        x = s[name + "_code"][page, :, idx % P].view(FP8).float() * s[name + "_scale"][page][..., None]
        res[name] = torch.where(held[..., None, None], x, torch.zeros_like(x)).to(DTYPES[case["dtype"]])
    return res


def run(s):
    kind = s["case"]["kind"]
    if own:
        from long_context_decode_02_b200 import lowram as L
        if kind == "append":
            L.paged_append(s["ctx"], s["pages"], s["k_new"], s["v_new"], cu_new=s["cu"],
                           max_new=s["max_new"], pos_base=s["base"])
            return _pools(s)
        if kind == "attend":
            L.paged_attend(s["ctx"], s["pages"], s["q"], s["out"], s["ws"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        L.paged_gather(s["ctx"], s["pages"], s["k_out"], s["v_out"], start=s["start"])
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"append": _plain_append, "attend": _plain_attend, "gather": _plain_gather}[kind](s)


# ------------------------------------------------------------------------------- work
def work(case):
    H, d, P, B = case["heads"], case["dim"], case["page"], case["batch"]
    es = 2 if case["dtype"] == "bf16" else 4
    lens = _lens(case)
    if case["kind"] == "append":
        n = sum(_new(case, lens))
        # rows in, codes out, a page's scales; three operations an element of the rotation, one
        # for the scale
        return {"bytes": 2 * n * H * d * (es + 1) + 8 * H * (n // P + B), "flops": 2 * n * H * d * 4}
    if case["kind"] == "attend":
        rows = B * case["queries"] * H * case["group"]
        pages = sum(-(-l // P) for l in lens)
        return {"bytes": 2 * sum(lens) * H * d + 8 * pages * H + 2 * rows * d * es + 4 * rows,
                "flops": 4 * case["queries"] * H * case["group"] * d * sum(lens)}
    n = case["count"]
    held = sum(max(0, min(n, l - a)) for l, a in zip(lens, _starts(case)))
    return {"bytes": 2 * H * d * (held + B * n * es), "flops": 2 * held * H * d}


# ------------------------------------------------------------------------------- 64 bits
def _value(codes):
    """The number that an e4m3 byte stands for, from its bits: sign, 4 exponent, 3 fraction."""
    c = codes.to(torch.int32)
    sign = 1.0 - 2.0 * (c >> 7).double()
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, f * 2.0 ** -9, (1.0 + f / 8.0) * torch.exp2((e - 7).double()))
    return sign * torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    H, d, P, B = case["heads"], case["dim"], case["page"], case["batch"]
    lens, table = s["lens"].tolist(), s["table"].long()
    if case["kind"] == "attend":
        G, nq = case["group"], case["queries"]
        out = torch.zeros(B, nq, H * G, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, nq, H * G), -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pg = table[b, :-(-n // P)]
            for h in range(H):
                k, v = ((_value(s[x + "_code"][pg, h]) * s[x + "_scale"][pg, h].double()[:, None, None])
                        .reshape(-1, d)[:n] for x in "kv")
                for j in range(nq):
                    m = n - nq + j + 1
                    if m <= 0:
                        continue
                    z = s["q"][b, j, h * G:(h + 1) * G].double() @ k[:m].T / d ** 0.5
                    out[b, j, h * G:(h + 1) * G] = torch.softmax(z, dim=-1) @ v[:m]
                    lse[b, j, h * G:(h + 1) * G] = torch.logsumexp(z, dim=-1)
        return {"out": out, "lse": lse}
    if case["kind"] == "gather":
        n = case["count"]
        res = {x: torch.zeros(B, n, H, d, dtype=torch.float64, device="cuda") for x in "kv"}
        for b, start in enumerate(s["start"].tolist()):
            m = max(0, min(n, lens[b] - start))
            pg = table[b, :-(-lens[b] // P)]
            for x in "kv":
                whole = _value(s[x + "_code"][pg]) * s[x + "_scale"][pg].double()[:, :, None, None]
                res[x][b, :m] = whole.transpose(1, 2).reshape(-1, H, d)[start:start + m]
        return res
    # append: code values before their rounding to 8 bits, and the scales
    new = _new(case, lens)
    code = {x: _value(s[x + "_code"]) for x in "kv"}
    scale = {x: s[x + "_scale"].double() for x in "kv"}
    freq = torch.tensor([THETA ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(new):
        first = lens[b] - n
        x1 = s["k_new"][at:at + n].double()
        pos = torch.arange(first, lens[b], device="cuda").double() + float(s["base"][b])
        z = torch.polar(torch.ones(n, d // 2, dtype=torch.float64, device="cuda"), pos[:, None] * freq)
        z = torch.complex(x1[..., : d // 2], x1[..., d // 2:]) * z[:, None]
        rows = {"k": torch.cat([z.real, z.imag], dim=-1), "v": s["v_new"][at:at + n].double()}
        at += n
        for p in range(first // P, -(-lens[b] // P) if n else 0):
            lo, hi = max(first, p * P), min(lens[b], (p + 1) * P)
            g = int(table[b, p])
            for x in "kv":
                r = rows[x][lo - first:hi - first].transpose(0, 1)          # [H][rows][d]
                top = r.abs().amax(dim=(1, 2)).tolist()
                e = [max(-64, math.ceil(math.log2(a / 448.0))) if a > 0 else -64 for a in top]
                was_e = scale[x][g].clone()
                to = torch.tensor([2.0 ** y for y in e], dtype=torch.float64, device="cuda")
                if lo > p * P:
                    to = torch.maximum(to, was_e)
                    code[x][g, :, :lo - p * P] *= (was_e / to)[:, None, None]
                scale[x][g] = to
                code[x][g, :, lo - p * P:hi - p * P] = r / to[:, None, None]
    return {"k_code": code["k"], "k_scale": scale["k"], "v_code": code["v"], "v_scale": scale["v"]}
