"""Paged serving with K and V held in 8 bits, as measured cases, each with its plain form.

A cache in pages keeps e4m3 codes and one f32 scale for each block: one page of one
KV head, K and V apart.  A step writes the new tokens' rows into it (``write``: q and
k rotated, k and v quantised, and the rows of the pages that changed read back as
what they now stand for), a program that moves requests elsewhere reads their rows
(``read``), and every layer attends the new tokens over what their request holds
(``attend``).

The writer's scale is the smallest power of two s >= 2^-64 with |x| <= 448 s for all
rows of the block; it grows with them, and codes that stand there already are moved
to the new one (exactly, but for those that become subnormal).  A block whose row 0
is written starts anew.

``run`` computes an operator with elementary torch operations, or with the library's
own entry points where ``own`` is true.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
LOWEST = 2.0 ** -64  # of the writer's scales
BASE = 500000.0


def _write(n_seq, new, longest, n_q, n_kv, hd, rot, layout, page, given, to, mix):
    return {"op": "write", "n_seq": n_seq, "new": new, "longest": longest, "n_q": n_q, "n_kv": n_kv, "hd": hd, "rot": rot,
            "layout": layout, "page": page, "given": given, "to": to, "mix": mix}


def _read(n_seq, longest, n_kv, hd, page, to, mix, ragged=True):
    return {"op": "read", "n_seq": n_seq, "longest": longest, "n_kv": n_kv, "hd": hd, "page": page, "to": to, "mix": mix,
            "ragged": ragged}


def _attend(n_seq, new, longest, n_q, n_kv, hd, page, dtype, mix, ragged=True, window=0, softcap=0.0, sinks=False):
    return {"op": "attend", "n_seq": n_seq, "new": new, "longest": longest, "n_q": n_q, "n_kv": n_kv, "hd": hd, "page": page,
            "dtype": dtype, "mix": mix, "ragged": ragged, "window": window, "softcap": softcap, "sinks": sinks}


def listed():
    return [
        # a decode step's rows: one token for each of 256 requests, into pages that hold rows already
        dict(_write(256, 1, 1024, 32, 8, 128, 128, "half", 16, "bf16", "bf16", 1), name="write decode"),
        # chunks of prompts, given in f32; half of each head carries positions; odd lengths
        dict(_write(29, 512, 4096, 10, 10, 64, 32, "interleaved", 64, "f32", "f16", 2), name="write chunks"),
        # one long prompt's q, k and v
        dict(_write(1, 8192, 8192, 32, 8, 128, 128, "half", 128, "bf16", "bf16", 3), name="write prompt"),
        # the rows of one short request, on their way to another cache
        dict(_read(1, 1023, 8, 128, 16, "bf16", 4, ragged=False), name="read short"),
        # requests of every length that leave the GPU's cache
        dict(_read(48, 16384, 8, 128, 16, "bf16", 5), name="read requests"),
        # the smallest call: one token of one request
        dict(_attend(1, 1, 1023, 32, 8, 128, 16, "bf16", 6, ragged=False), name="attend one token"),
        # a decode step over requests of every length
        dict(_attend(64, 1, 16384, 32, 8, 128, 16, "bf16", 7), name="attend decode"),
        # few requests with long contexts, 16 query heads for each KV head
        dict(_attend(4, 1, 131072, 128, 8, 128, 64, "f16", 8, ragged=False), name="attend long"),
        # four drafted tokens checked at once for each of 32 requests
        dict(_attend(32, 4, 4096, 32, 8, 128, 32, "bf16", 9), name="attend drafts"),
        # chunks of several prompts with a sliding window, capped scores and sinks
        dict(_attend(7, 700, 5000, 16, 4, 64, 64, "f16", 10, window=1024, softcap=30.0, sinks=True), name="attend window"),
        # a chunk of a long prompt: the compute-bound end
        dict(_attend(1, 4096, 32768, 32, 8, 128, 128, "bf16", 11, ragged=False), name="attend prompt"),
    ]


def _spread(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["write", "write", "read", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    hd = rng.choice([64, 128, 128])
    n_kv = rng.choice([1, 2, 4, 8, 10])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "write":
        n_seq = _spread(rng, 1, 256)
        rot = rng.choice([hd, hd, hd // 2, hd // 4, hd // 2 + 6])
        return _write(n_seq, _spread(rng, 1, max(1, 8192 // n_seq)), _spread(rng, 16, max(16, min(16384, 262144 // n_seq))),
                      n_kv * min(group, 4 if n_kv < 10 else 2), n_kv, hd, rot, rng.choice(["half", "interleaved"]), page,
                      rng.choice(["f32", dtype]), dtype, mix)
    if op == "read":
        longest = _spread(rng, 1, 65536)
        return _read(_spread(rng, 1, max(1, min(128, (1 << 22) // (n_kv * longest)))), longest, n_kv, hd, page,
                     rng.choice(["f32", "f16", "bf16"]), mix, ragged=rng.random() < 0.7)
    longest = _spread(rng, 1, 65536)
    n_seq = _spread(rng, 1, max(1, min(128, (1 << 22) // (n_kv * longest))))
    rows = max(1, min(4096, longest, (1 << 32) // (longest * n_seq * n_kv * group)))  # scores of the padded batch
    new = _spread(rng, 1, rows)
    return _attend(n_seq, new, longest, n_kv * group, n_kv, hd, page, dtype, mix, ragged=rng.random() < 0.7,
                   window=rng.choice([0, 0, _spread(rng, 1, longest)]), softcap=rng.choice([0.0, 0.0, 30.0]), sinks=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """Rows that each request holds before the step, and its new tokens (host arrays)."""
    r = np.random.RandomState(case["mix"])
    n, longest = case["n_seq"], case["longest"]
    if case["op"] == "read":
        total = r.randint(1, longest + 1, n) if case["ragged"] else np.full(n, longest)
        return total, np.zeros_like(total)
    new = case["new"]
    if case["op"] == "attend":
        total = r.randint(new, max(new, longest) + 1, n) if case["ragged"] else np.full(n, max(new, longest))
        fresh = r.randint(1, new + 1, n) if case["ragged"] and new > 8 else np.full(n, new)
        return total - fresh, fresh
    if n == 1:
        return np.zeros(1, np.int64), np.full(1, new)
    return r.randint(0, longest + 1, n), r.randint(1, new + 1, n)


def _table(total, page, g, device):
    """Block table of shuffled pages, and how many pages the pool has."""
    most = -(-total // page)
    width, n_pages = int(most.max()) + 1, int(most.sum()) + 5
    order = torch.randperm(n_pages, generator=g, device=device, dtype=torch.int32)
    taken = torch.arange(width, device=device)[None, :] < torch.from_numpy(most).to(device)[:, None]
    table = torch.full((len(total), width), -1, dtype=torch.int32, device=device)
    table[taken] = order[: int(most.sum())]
    return table, n_pages


def _ints(a, device):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).to(device)


def _cu(n):
    return np.concatenate([[0], np.cumsum(n)])


def _scale_for(top):
    """The writer's scale for blocks whose largest value is `top` (f32): 448 = 0.875 * 2^9."""
    m, e = torch.frexp(top)
    e = e - torch.where(m <= 0.875, 9, 8).to(e.dtype)
    s = ((e.clamp(-64, 64) + 127) << 23).view(torch.float32)  # 2^e by its bits: no power function is exact enough
    return torch.where(top > 0, s, torch.full_like(s, LOWEST))


def _pages(shape, g, device, sigma):
    """Codes and scales of a pool whose blocks differ in size, as layers' keys and values do."""
    codes = torch.empty(shape, dtype=E4M3, device=device)
    scale = torch.empty(shape[:2], dtype=torch.float32, device=device)
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for a in range(0, shape[0], step):
        b = min(shape[0], a + step)
        x = torch.randn((b - a, *shape[1:]), generator=g, device=device).mul_(sigma)
        x *= torch.exp(torch.rand((b - a, shape[1], 1, 1), generator=g, device=device) * 1.4 - 0.7)
        scale[a:b] = _scale_for(x.abs().amax((2, 3)))
        codes[a:b] = (x / scale[a:b, :, None, None]).to(E4M3)
    return codes, scale


def _frequencies(case):
    return BASE ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(seed)
    s = dict(case)
    held, fresh = _lengths(case)
    total, page, n_kv, hd = held + fresh, case["page"], case["n_kv"], case["hd"]
    s["max_len"], s["max_new"], s["tokens"] = int(total.max()), int(fresh.max()), int(fresh.sum())
    s["error"] = torch.zeros(1, dtype=torch.int32, device=device)
    s["table"], n_pages = _table(total, page, g, device)
    s["seq_len"] = _ints(total, device)
    # keys carry channels of different size, as rotated keys do
    sigma = torch.exp(torch.rand(hd, generator=g, device=device) * 1.4 - 0.7)
    s["k_pages"], s["k_scale"] = _pages((n_pages, n_kv, page, hd), g, device, sigma)
    s["v_pages"], s["v_scale"] = _pages((n_pages, n_kv, page, hd), g, device, torch.ones(hd, device=device))
    if case["op"] == "read":
        s["start"], rows = None, total
    elif case["op"] == "write":
        s["start"], rows = _ints(held // page * page, device), total - held // page * page
    if case["op"] != "attend":
        s["cu_rows"], s["rows"] = _ints(_cu(rows), device), int(rows.sum())
    if case["op"] == "read":
        return s
    s["cu_new"] = _ints(_cu(fresh), device)
    if case["op"] == "write":
        seq = np.repeat(np.arange(case["n_seq"]), fresh)
        pos = np.concatenate([np.arange(a, b) for a, b in zip(held, total)])
        at, off = torch.from_numpy(pos // page).to(device), torch.from_numpy(pos % page).to(device)
        s["positions"] = _ints(pos, device)
        s["slots"] = (s["table"][torch.from_numpy(seq).to(device), at].long() * page + off).to(torch.int32)
        b = np.flatnonzero(held % page)
        s["tails"] = s["table"][torch.from_numpy(b).to(device), torch.from_numpy(held[b] // page).to(device)].long()
        s["tail_rows"] = torch.from_numpy(held[b] % page).to(device)
        given = DTYPES[case["given"]]
        qkv = torch.randn(s["tokens"], case["n_q"] + 2 * n_kv, hd, generator=g, device=device)
        qkv[:, case["n_q"]:] *= torch.exp(torch.rand(s["tokens"], 1, 1, generator=g, device=device) * 1.4 - 0.7)
        qkv = qkv.to(given)  # one projection's output: q, k and v are its slices
        s["q"], s["k"], s["v"] = qkv[:, : case["n_q"]], qkv[:, case["n_q"]: case["n_q"] + n_kv], qkv[:, case["n_q"] + n_kv:]
        s["freq"] = _frequencies(case).to(device)
        return s
    s["q"] = torch.randn(s["tokens"], case["n_q"], hd, generator=g, device=device, dtype=DTYPES[case["dtype"]])
    s["sink"] = torch.randn(case["n_q"], generator=g, device=device) if case["sinks"] else None
    s["scale"] = 1.0 / math.sqrt(hd)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _own(s)
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)


def _own(s):
    import kv_cache_decode_attention_gb300 as kvd

    cache = kvd.PagedKvCache.of(s["k_pages"], s["v_pages"], s["table"], s["seq_len"], error=s["error"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"])
    if s["op"] == "read":
        return kvd.paged_read(cache, s["cu_rows"], s["rows"], dtype=DTYPES[s["to"]])
    if s["op"] == "write":
        plan = kvd.PagedPlan(s["cu_new"], s["seq_len"], None, s["positions"], s["slots"])
        q_out = torch.empty(s["q"].shape, dtype=DTYPES[s["to"]], device=s["q"].device)
        q = kvd.paged_append(cache, plan, s["k"], s["v"], q=s["q"], q_out=q_out,
                             rope=kvd.RopeTable(s["rot"], layout=s["layout"], base=BASE))
        k, v = kvd.paged_read(cache, s["cu_rows"], s["rows"], start=s["start"], dtype=DTYPES["bf16"])
        return {"q": q, "k": k, "v": v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    plan = kvd.PagedPlan(s["cu_new"], s["seq_len"])
    return kvd.paged_attention(s["q"], cache, plan, scale=s["scale"], window=s["window"], softcap=s["softcap"], sinks=s["sink"])


def _rotate(x, positions, freq, layout):
    """f32 result of the rotation of x [tokens, heads, hd]; the angles are taken in f64."""
    n = freq.numel()
    angle = positions.double()[:, None] * freq[None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    x = x.float()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if layout == "interleaved" else (x[..., :n], x[..., n:2 * n])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if layout == "interleaved" else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _rows_of(s, start):
    """Request and position of each row that cu_rows and start name."""
    cu = s["cu_rows"].long()
    seq = torch.repeat_interleave(torch.arange(s["n_seq"], device=cu.device), cu[1:] - cu[:-1], output_size=s["rows"])
    pos = torch.arange(s["rows"], device=cu.device) - cu[seq]
    return seq, pos if start is None else pos + start.long()[seq]


def _plain_read(s, start=None, to=None):
    seq, pos = _rows_of(s, start)
    page, off = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    out = []
    for codes, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])):
        # (indexed as bytes: codes of 8 bits have no gather of their own)
        x = codes.view(torch.uint8)[page, :, off].view(E4M3).float()
        out.append((x * scale[page][:, :, None]).to(DTYPES[to or s["to"]]))
    return tuple(out)


def _plain_store(s, codes, scale, x):
    """Rows x (f32) to their slots; the blocks' scales grow and their codes move with them."""
    size = s["page"]
    page, off = s["slots"].long() // size, s["slots"].long() % size
    raw = codes.view(torch.uint8)
    grown = _scale_for(torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax"))
    # pages that hold rows before the new ones: no scale shrinks, and what stands there moves to the new one
    at, rows = s["tails"], s["tail_rows"]
    grown[at] = torch.maximum(grown[at], scale[at])
    moved = (raw[at].view(E4M3).float() * (scale[at] / grown[at])[:, :, None, None]).to(E4M3)
    stay = (torch.arange(size, device=x.device)[None, :] < rows[:, None])[:, None, :, None]
    raw[at] = torch.where(stay, moved.view(torch.uint8), raw[at])
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    scale.copy_(torch.where(touched[:, None], grown, scale))
    raw[page, :, off] = (x / scale[page][:, :, None]).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _plain_write(s):
    q = _rotate(s["q"], s["positions"], s["freq"], s["layout"]).to(DTYPES[s["to"]])
    _plain_store(s, s["k_pages"], s["k_scale"], _rotate(s["k"], s["positions"], s["freq"], s["layout"]))
    _plain_store(s, s["v_pages"], s["v_scale"], s["v"].float())
    k, v = _plain_read(s, s["start"], "bf16")
    return {"q": q, "k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_attend(s):
    q, page, device = s["q"], s["page"], s["q"].device
    n_kv, group, hd = s["n_kv"], s["n_q"] // s["n_kv"], s["hd"]
    n_seq, width = s["n_seq"], -(-s["max_len"] // page)
    pages = s["table"][:, :width].long().clamp_min(0)

    def rows(codes, scale):
        x = codes.view(torch.uint8)[pages].view(E4M3).float() * scale[pages][..., None, None]
        return x.transpose(1, 2).reshape(n_seq, n_kv, width * page, hd)

    k, v = rows(s["k_pages"], s["k_scale"]), rows(s["v_pages"], s["v_scale"])
    cu, total = s["cu_new"].long(), s["seq_len"].long()
    fresh = cu[1:] - cu[:-1]
    i = torch.arange(s["max_new"], device=device)
    row = (cu[:-1, None] + i[None, :]).clamp_max(s["tokens"] - 1)
    x = q[row].float().reshape(n_seq, s["max_new"], n_kv, group, hd).permute(0, 2, 3, 1, 4).reshape(n_seq, n_kv, group * s["max_new"], hd)
    score = torch.matmul(x, k.transpose(-1, -2)).mul_(s["scale"]).reshape(n_seq, n_kv, group, s["max_new"], width * page)
    if s["softcap"] > 0:
        score = torch.tanh(score / s["softcap"]) * s["softcap"]
    pos = (total - fresh)[:, None] + i[None, :]
    at = torch.arange(width * page, device=device)
    seen = at[None, None, :] <= pos[:, :, None]
    if s["window"] > 0:
        seen &= at[None, None, :] > pos[:, :, None] - s["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].reshape(1, n_kv, group, 1, 1)
        top = torch.maximum(top, sink)
    score.sub_(top).exp_()
    below = score.sum(-1, keepdim=True)
    if s["sink"] is not None:
        below = below + torch.exp(sink - top)
    o = torch.matmul(score.reshape(n_seq, n_kv, group * s["max_new"], -1), v).reshape(n_seq, n_kv, group, s["max_new"], hd) / below
    o = o.permute(0, 3, 1, 2, 4).reshape(n_seq, s["max_new"], n_kv * group, hd)
    return o[i[None, :] < fresh[:, None]].to(q.dtype)


# ------------------------------------------------------------------ bounds and the definition


def work(case):
    held, fresh = _lengths(case)
    total, t, page, n_kv, hd = held + fresh, int(fresh.sum()), case["page"], case["n_kv"], case["hd"]
    if case["op"] == "read":
        rows, blocks = int(total.sum()), int((-(-total // page)).sum())
        return {"bytes": 2 * rows * n_kv * hd * (1 + DTYPES[case["to"]].itemsize) + 8 * blocks * n_kv + 4 * blocks, "flops": 2 * rows * n_kv * hd}
    if case["op"] == "write":
        back = int((total - held // page * page).sum())           # rows read back
        blocks = int((-(-total // page) - held // page).sum())    # pages touched
        given, to = DTYPES[case["given"]].itemsize, DTYPES[case["to"]].itemsize
        into = t * (case["n_q"] * (given + to) + 2 * n_kv * (given + 1)) * hd + 8 * t + 8 * blocks * n_kv
        return {"bytes": into + 2 * back * n_kv * hd * 2 + 2 * (back - t) * n_kv * hd, "flops": 3 * t * (case["n_q"] + 2 * n_kv) * hd}
    window = case["window"] or 1 << 40
    rows = int(np.minimum(total, fresh + window - 1).sum())  # cached rows that some new token sees
    pairs = int(sum(np.minimum(np.arange(a, b) + 1, window).sum() for a, b in zip(held, total)))
    return {"bytes": 2 * rows * n_kv * hd + 2 * t * case["n_q"] * hd * DTYPES[case["dtype"]].itemsize + -(-rows // page) * (4 + 8 * n_kv),
            "flops": 4 * pairs * case["n_q"] * hd}


def _exact_turn(x, positions, case):
    """The rotation as a complex product in 64 bits."""
    f = _frequencies(case)
    n = f.numel()
    unit = torch.polar(torch.ones(len(positions), n, dtype=torch.float64), positions.double().cpu()[:, None] * f).to(x.device)[:, None]
    out = x.double().clone()
    if case["layout"] == "interleaved":
        z = torch.view_as_complex(out[..., : 2 * n].reshape(*out.shape[:-1], n, 2).contiguous()) * unit
        out[..., : 2 * n] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(out[..., :n], out[..., n: 2 * n]) * unit
        out[..., :n], out[..., n: 2 * n] = z.real, z.imag
    return out


def _power(e):
    """2^e in 64 bits, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_code(x):
    """x to the nearest of the e4m3 numbers (ties to even, 448 at most), by its exponent."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
    step = _power(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    held, fresh = _lengths(case)
    total, page, n_kv, hd = held + fresh, case["page"], case["n_kv"], case["hd"]
    table = s["table"].cpu().numpy()

    def pages_of(codes, scale, b, first, last):
        """Rows [first, last) of request b in 64 bits, [n_kv, rows, hd]."""
        p = torch.from_numpy(table[b, first // page: -(-last // page)].astype(np.int64)).to(codes.device)
        x = codes.view(torch.uint8)[p].view(E4M3).double() * scale[p].double()[:, :, None, None]
        return x.transpose(0, 1).reshape(n_kv, -1, hd)[:, first - first // page * page: last - first // page * page]

    if case["op"] == "read":
        if int(total.sum()) > 1 << 19:
            return None
        return tuple(torch.cat([pages_of(c, z, b, 0, int(total[b])).transpose(0, 1) for b in range(case["n_seq"])])
                     for c, z in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
    if case["op"] == "write":
        q, k = _exact_turn(s["q"], s["positions"], case), _exact_turn(s["k"], s["positions"], case)
        out = {"q": q}
        for name, x in (("k", k), ("v", s["v"].double())):
            codes, scale = s[name + "_pages"], s[name + "_scale"].double().clone()
            rows, t0 = [], 0
            for b in range(case["n_seq"]):
                first, last = int(held[b]), int(total[b])
                for p0 in range(first // page * page, last, page):
                    at = int(table[b, p0 // page])
                    lo, hi = max(first, p0), min(last, p0 + page)
                    new = x[t0 + lo - first: t0 + hi - first].transpose(0, 1)
                    top = new.abs().amax((1, 2))
                    need = _power(torch.round(torch.log2(top / 448.0).clamp_min(-64)) - 1)  # too small, then right
                    for _ in range(2):
                        need = torch.where(top > 448.0 * need, 2.0 * need, need)
                    need = need.clamp_min(LOWEST)
                    old = scale[at].clone()
                    size = torch.maximum(old, need) if lo > p0 else need
                    scale[at] = size
                    block = _exact_code(new / size[:, None, None])
                    if lo > p0:
                        stay = codes[at, :, : lo - p0].double()
                        block = torch.cat([_exact_code(stay * (old / size)[:, None, None]), block], 1)
                    rows.append((block * size[:, None, None]).transpose(0, 1))
                t0 += last - first
            out[name], out[name + "_scale"] = torch.cat(rows), scale
        return {n: out[n] for n in ("q", "k", "v", "k_scale", "v_scale")}
    group = case["n_q"] // n_kv
    out = torch.empty(s["tokens"], case["n_q"], hd, dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["n_seq"]):
        n, last = int(fresh[b]), int(total[b])
        p = torch.from_numpy(table[b, : -(-last // page)].astype(np.int64)).to("cuda")
        pos = torch.arange(last - n, last, device="cuda")[:, None]
        at = torch.arange(last, device="cuda")[None, :]
        hidden = (at > pos) | ((at <= pos - case["window"]) if case["window"] else (at < 0))
        for h in range(n_kv):
            k, v = ((c.view(torch.uint8)[p, h].view(E4M3).double() * z[p, h].double()[:, None, None]).reshape(-1, hd)[:last]
                    for c, z in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            for j in range(h * group, (h + 1) * group):
                w = (s["q"][t0:t0 + n, j].double() @ k.T) / math.sqrt(hd)
                if case["softcap"]:
                    w = case["softcap"] * torch.tanh(w / case["softcap"])
                w = w.masked_fill(hidden, -math.inf)
                if s["sink"] is not None:
                    w = torch.cat([w, s["sink"][j].double().expand(n, 1)], 1)
                w = torch.softmax(w, -1)[:, :last]
                out[t0:t0 + n, j] = w @ v
        t0 += n
    return out
