"""The paged serving operators as measured cases, each with its plain form.

One step of a paged server is: place the new tokens of every request
(``plan``), rotate q and k (``rope``) or rotate and write K and V into their
pages in one go (``append``), and attend the new tokens over everything their
request holds (``attend``).  ``run`` computes an operator with elementary torch
operations, or with the library's own entry points where ``own`` is true.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
YARN = {"factor": 8.0, "original_len": 4096.0, "beta_fast": 32.0, "beta_slow": 1.0}
BANDS = {"factor": 8.0, "original_len": 8192.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0}
LINEAR = {"factor": 4.0}
NTK = {"factor": 4.0}


def _plan(n_seq, page, longest, new, finished, mix):
    return {"op": "plan", "n_seq": n_seq, "page": page, "longest": longest, "new": new, "finished": finished, "mix": mix}


def _rope(tokens, n_q, n_kv, hd, rot, layout, scaling, dtype, far):
    return {"op": "rope", "tokens": tokens, "n_q": n_q, "n_kv": n_kv, "hd": hd, "rot": rot, "layout": layout,
            "scaling": scaling, "dtype": dtype, "far": far}


def _append(n_seq, new, longest, n_q, n_kv, hd, rot, layout, scaling, page, dtype, given, mix):
    return {"op": "append", "n_seq": n_seq, "new": new, "longest": longest, "n_q": n_q, "n_kv": n_kv, "hd": hd, "rot": rot,
            "layout": layout, "scaling": scaling, "page": page, "dtype": dtype, "given": given, "mix": mix}


def _attend(n_seq, new, longest, n_q, n_kv, hd, page, dtype, mix, ragged=True, window=0, softcap=0.0, sinks=False):
    return {"op": "attend", "n_seq": n_seq, "new": new, "longest": longest, "n_q": n_q, "n_kv": n_kv, "hd": hd, "page": page,
            "dtype": dtype, "mix": mix, "ragged": ragged, "window": window, "softcap": softcap, "sinks": sinks}


def listed():
    return [
        # one decode step of the ragged serving batch: a token for each of 256 requests, a few of which have just finished
        dict(_plan(256, 16, 16384, 1, 0.03, 1), name="plan decode"),
        # a step that admits prompts: up to 256 new tokens for each of 500 requests
        dict(_plan(500, 64, 8192, 256, 0.25, 2), name="plan chunks"),
        # the rows of one new token of one request, f32, on their way to the contiguous cache
        dict(_rope(1, 32, 8, 128, 128, "interleaved", "none", "f32", 16384), name="rope one token"),
        # a long prompt's q and k, positions scaled to 8 times the trained length
        dict(_rope(8192, 32, 8, 128, 128, "half", "yarn", "bf16", 131072), name="rope prompt"),
        # a decode step's rows into pages: one token for each of 256 requests
        dict(_append(256, 1, 1024, 32, 8, 128, 128, "half", "none", 16, "bf16", "bf16", 3), name="append decode"),
        # chunks of prompts into pages; half of each head carries positions, rows come in f32
        dict(_append(29, 512, 4096, 10, 10, 128, 64, "interleaved", "linear", 64, "f16", "f32", 4), name="append chunks"),
        # the smallest call: one token of one request
        dict(_attend(1, 1, 1023, 32, 8, 128, 16, "bf16", 5, ragged=False), name="attend one token"),
        # a decode step over requests of every length
        dict(_attend(64, 1, 16384, 32, 8, 128, 16, "bf16", 6), name="attend decode"),
        # few requests with long contexts, 16 query heads for each KV head
        dict(_attend(4, 1, 131072, 128, 8, 128, 64, "f16", 7, ragged=False), name="attend long"),
        # four drafted tokens checked at once for each of 32 requests
        dict(_attend(32, 4, 4096, 32, 8, 128, 32, "bf16", 8), name="attend drafts"),
        # chunks of several prompts with a sliding window, capped scores and sinks
        dict(_attend(7, 700, 5000, 16, 4, 64, 64, "f16", 9, window=1024, softcap=30.0, sinks=True), name="attend window"),
        # a chunk of a long prompt: the compute-bound end
        dict(_attend(1, 4096, 32768, 32, 8, 128, 128, "bf16", 10, ragged=False), name="attend prompt"),
    ]


def _spread(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "append", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 20)
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    hd = rng.choice([64, 128, 128])
    rot = rng.choice([hd, hd, hd // 2, hd // 4, hd // 2 + 6])
    layout = rng.choice(["half", "interleaved"])
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
    n_kv = rng.choice([1, 2, 4, 8, 10])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    if op == "plan":
        return _plan(_spread(rng, 1, 500), page, _spread(rng, 16, 16384), _spread(rng, 1, 256), rng.choice([0.0, 0.05, 0.3]), mix)
    if op == "rope":
        group = min(group, 40 // n_kv)
        return _rope(_spread(rng, 1, 8192), n_kv * group, n_kv, hd, rot, layout, scaling, rng.choice(["f32", dtype]) if n_kv * group <= 20 else dtype,
                     _spread(rng, 1024, 1 << 20))
    if op == "append":
        n_seq = _spread(rng, 1, 256)
        return _append(n_seq, _spread(rng, 1, max(1, 8192 // n_seq)), _spread(rng, 16, max(16, min(16384, 262144 // n_seq))), n_kv * min(group, 2), n_kv, hd, rot, layout, scaling, page,
                       dtype, rng.choice(["f32", dtype]), mix)
    longest = _spread(rng, 1, 65536)
    n_seq = _spread(rng, 1, max(1, min(128, (1 << 22) // (n_kv * longest))))
    rows = max(1, min(4096, longest, (1 << 32) // (longest * n_seq * n_kv * group)))  # scores of the padded batch
    new = _spread(rng, 1, rows)
    return _attend(n_seq, new, longest, n_kv * group, n_kv, hd, page, dtype, mix, ragged=rng.random() < 0.7,
                   window=rng.choice([0, 0, _spread(rng, 1, longest)]), softcap=rng.choice([0.0, 0.0, 30.0]), sinks=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs


def _lengths(case):
    """Rows that each request holds before the step, rows it keeps, and its new tokens (host arrays)."""
    r = np.random.RandomState(case["mix"])
    n, new, longest = case["n_seq"], case["new"], case["longest"]
    if case["op"] == "attend":
        total = r.randint(new, max(new, longest) + 1, n) if case["ragged"] else np.full(n, max(new, longest))
        fresh = r.randint(1, new + 1, n) if case["ragged"] and new > 8 else np.full(n, new)
        return total - fresh, total - fresh, fresh
    held = r.randint(1, longest + 1, n)
    fresh = r.randint(1, new + 1, n)
    done = r.uniform(size=n) < case.get("finished", 0.0)
    return held, np.where(done, 0, held), fresh


def _tables(held, total, page, g, device):
    """Block table of shuffled pages for the rows held, the stack of free pages and its height."""
    has, most = -(-held // page), -(-np.maximum(held, total) // page)
    width = int(most.max()) + 1
    spare = int(np.maximum(most - has, 0).sum()) + 5
    n_pages = int(has.sum()) + spare
    order = torch.randperm(n_pages, generator=g, device=device, dtype=torch.int32)
    taken = torch.arange(width, device=device)[None, :] < torch.from_numpy(has).to(device)[:, None]
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=device)
    table[taken] = order[: int(has.sum())]
    free = torch.zeros(n_pages, dtype=torch.int32, device=device)
    free[:spare] = order[int(has.sum()):]
    return table, free, spare, n_pages


def _ints(a, device):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).to(device)


def _frequencies(case):
    """Angle per position of each rotated pair (f64, host) and the factor on cos and sin, with the scaling of long contexts."""
    rot, kind = case["rot"], case["scaling"]
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    base = 10000.0
    if kind == "ntk":
        base = base * NTK["factor"] ** (rot / (rot - 2))
    f = base ** (-i / rot)
    if kind == "linear":
        return f / LINEAR["factor"], 1.0
    if kind == "yarn":
        def at(turns):
            return rot * math.log(YARN["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))

        low, high = max(math.floor(at(YARN["beta_fast"])), 0), min(math.ceil(at(YARN["beta_slow"])), rot - 1)
        ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f / YARN["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(YARN["factor"]) + 1.0
    if kind == "bands":
        wave = BANDS["original_len"] * f / (2 * math.pi)
        blend = ((wave - BANDS["low_freq_factor"]) / (BANDS["high_freq_factor"] - BANDS["low_freq_factor"])).clamp(0, 1)
        return f / BANDS["factor"] * (1 - blend) + f * blend, 1.0
    return f, 1.0


def _rope_options(case):
    more = {"none": {}, "linear": LINEAR, "ntk": NTK, "yarn": YARN, "bands": BANDS}[case["scaling"]]
    return dict(rot_dim=case["rot"], layout=case["layout"], scaling=case["scaling"], base=10000.0, **more)


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(seed)
    s = dict(case)

    def normal(*shape, dtype, sigma=None):
        x = torch.randn(*shape, generator=g, device=device, dtype=dtype)
        return x if sigma is None else x.mul_(sigma.to(dtype))

    if case["op"] == "rope":
        t, dt = case["tokens"], DTYPES[case["dtype"]]
        qkv = normal(t, case["n_q"] + case["n_kv"], case["hd"], dtype=dt)  # one projection's output: q and k are its slices
        s["q"], s["k"] = qkv[:, : case["n_q"]], qkv[:, case["n_q"]:]
        start = int(torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=device))
        s["positions"] = torch.arange(start, start + t, device=device, dtype=torch.int32)
        s["freq"], s["factor"] = _frequencies(case)
        s["freq"] = s["freq"].to(device)
        s["rope"] = _rope_options(case)
        return s
    held, keep, fresh = _lengths(case)
    total = keep + fresh
    s["max_len"], s["max_new"], s["tokens"] = int(total.max()), int(fresh.max()), int(fresh.sum())
    s["error"] = torch.zeros(1, dtype=torch.int32, device=device)
    if case["op"] == "plan":
        s["table"], s["free"], spare, _ = _tables(held, total, case["page"], g, device)
        s["held"], s["keep"], s["new_len"] = _ints(held, device), _ints(keep, device), _ints(fresh, device)
        s["n_free"] = torch.tensor([spare], dtype=torch.int32, device=device)
        return s
    page, dt = case["page"], DTYPES[case["dtype"]]
    s["table"], s["free"], spare, n_pages = _tables(total, total, page, g, device)
    s["n_free"] = torch.tensor([spare], dtype=torch.int32, device=device)
    s["seq_len"] = _ints(total, device)
    s["cu_new"] = _ints(np.concatenate([[0], np.cumsum(fresh)]), device)
    t, hd, n_kv = s["tokens"], case["hd"], case["n_kv"]
    if case["op"] == "append":
        seq = np.repeat(np.arange(case["n_seq"]), fresh)
        pos = np.concatenate([np.arange(a, b) for a, b in zip(keep, total)])
        s["positions"] = _ints(pos, device)
        at, off = torch.from_numpy(pos // page).to(device), torch.from_numpy(pos % page).to(device)
        s["slots"] = (s["table"][torch.from_numpy(seq).to(device), at].long() * page + off).to(torch.int32)
        given = DTYPES[case["given"]]
        qkv = normal(t, case["n_q"] + 2 * n_kv, hd, dtype=given)
        s["q"], s["k"], s["v"] = qkv[:, : case["n_q"]], qkv[:, case["n_q"]: case["n_q"] + n_kv], qkv[:, case["n_q"] + n_kv:]
        s["k_pages"] = torch.zeros(n_pages, n_kv, page, hd, device=device, dtype=dt)
        s["v_pages"] = torch.zeros(n_pages, n_kv, page, hd, device=device, dtype=dt)
        s["freq"], s["factor"] = _frequencies(case)
        s["freq"] = s["freq"].to(device)
        s["rope"] = _rope_options(case)
        return s
    # keys carry channels of different size, as rotated keys do
    sigma = torch.exp(torch.rand(hd, generator=g, device=device) * 1.4 - 0.7)
    s["k_pages"] = normal(n_pages, n_kv, page, hd, dtype=dt, sigma=sigma)
    s["v_pages"] = normal(n_pages, n_kv, page, hd, dtype=dt)
    s["q"] = normal(t, case["n_q"], hd, dtype=dt)
    s["sink"] = normal(case["n_q"], dtype=torch.float32) if case["sinks"] else None
    s["scale"] = 1.0 / math.sqrt(hd)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _own(s)
    return {"plan": _plain_plan, "rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


def _own(s):
    import kv_cache_decode_attention_gb300 as kvd

    if s["op"] == "rope":
        return kvd.rope(s["q"], s["k"], s["positions"], kvd.RopeTable(**s["rope"]))
    if s["op"] == "plan":
        cache = kvd.PagedKvCache.of(None, None, s["table"], s["held"], s["free"], s["n_free"], error=s["error"], page_size=s["page"])
        p = kvd.paged_plan(cache, s["new_len"], s["tokens"], keep_len=s["keep"], advance=False)
        return {"table": cache.block_table, "free": cache.free_pages, "n_free": p.n_free, "seq_len": p.seq_len, "cu_new": p.cu_new,
                "positions": p.positions, "slots": p.slots}
    cache = kvd.PagedKvCache.of(s["k_pages"], s["v_pages"], s["table"], s["seq_len"], s["free"], s["n_free"], error=s["error"])
    if s["op"] == "append":
        plan = kvd.PagedPlan(s["cu_new"], s["seq_len"], s["n_free"], s["positions"], s["slots"])
        q = kvd.paged_append(cache, plan, s["k"], s["v"], q=s["q"], rope=kvd.RopeTable(**s["rope"]))
        return {"q": q, "k_pages": cache.k, "v_pages": cache.v}
    plan = kvd.PagedPlan(s["cu_new"], s["seq_len"])
    return kvd.paged_attention(s["q"], cache, plan, scale=s["scale"], window=s["window"], softcap=s["softcap"], sinks=s["sink"])


def _plain_plan(s):
    page, device = s["page"], s["table"].device
    held, keep, new = s["held"].long(), s["keep"].long(), s["new_len"].long()
    total = keep + new
    has, after = (held + page - 1) // page, (total + page - 1) // page
    col = torch.arange(s["table"].shape[1], device=device)[None, :]
    table, free = s["table"], torch.cat([s["free"], s["free"][:1]])  # a place more, for what is not pushed
    # pages past a request's new end go on the stack, in order of requests and of pages
    gone = (col >= after[:, None]) & (col < has[:, None])
    at = s["n_free"].long() + torch.cumsum(gone.reshape(-1).long(), 0) - 1
    free[torch.where(gone.reshape(-1), at, free.numel() - 1)] = table.reshape(-1)
    free = free[:-1]
    top = s["n_free"].long() + gone.sum()
    # missing ones come off its top in the same order
    want = (col >= has[:, None]) & (col < after[:, None])
    take = (top - torch.cumsum(want.reshape(-1).long(), 0)).clamp_min(0)
    table = torch.where(want, free[take].reshape(table.shape), table)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=device), torch.cumsum(new, 0)])
    seq = torch.repeat_interleave(torch.arange(len(new), device=device), new, output_size=s["tokens"])
    pos = keep[seq] + torch.arange(s["tokens"], device=device) - cu[seq]
    slots = table[seq, pos // page].long() * page + pos % page
    i32 = torch.int32
    return {"table": table, "free": free, "n_free": (top - want.sum()).reshape(1).to(i32), "seq_len": total.to(i32), "cu_new": cu.to(i32),
            "positions": pos.to(i32), "slots": slots.to(i32)}


def _rotate(x, positions, freq, factor, layout):
    """f32 result of the rotation of x [tokens, heads, hd]; the angles are taken in f64."""
    n = freq.numel()
    angle = positions.double()[:, None] * freq[None, :]
    cos, sin = (torch.cos(angle) * factor).float()[:, None, :], (torch.sin(angle) * factor).float()[:, None, :]
    x = x.float()
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if layout == "interleaved" else (x[..., :n], x[..., n:2 * n])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if layout == "interleaved" else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _plain_rope(s):
    return tuple(_rotate(x, s["positions"], s["freq"], s["factor"], s["layout"]).to(x.dtype) for x in (s["q"], s["k"]))


def _plain_append(s):
    dt = s["k_pages"].dtype
    q = _rotate(s["q"], s["positions"], s["freq"], s["factor"], s["layout"]).to(dt)
    k = _rotate(s["k"], s["positions"], s["freq"], s["factor"], s["layout"]).to(dt)
    page, off = s["slots"].long() // s["page"], s["slots"].long() % s["page"]
    s["k_pages"][page, :, off] = k
    s["v_pages"][page, :, off] = s["v"].to(dt)
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(s):
    q, page, device = s["q"], s["page"], s["q"].device
    n_kv, group, hd = s["n_kv"], s["n_q"] // s["n_kv"], s["hd"]
    n_seq, width = s["n_seq"], -(-s["max_len"] // page)
    pages = s["table"][:, :width].long().clamp_min(0)
    k = s["k_pages"][pages].transpose(1, 2).reshape(n_seq, n_kv, width * page, hd).float()
    v = s["v_pages"][pages].transpose(1, 2).reshape(n_seq, n_kv, width * page, hd).float()
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
    if case["op"] == "rope":
        values = case["tokens"] * (case["n_q"] + case["n_kv"]) * case["hd"]
        return {"bytes": 2 * values * DTYPES[case["dtype"]].itemsize + 4 * case["tokens"], "flops": 3 * values}
    held, keep, fresh = _lengths(case)
    total, t = keep + fresh, int(fresh.sum())
    if case["op"] == "plan":
        has, after = -(-held // case["page"]), -(-total // case["page"])
        moved = int(np.abs(after - has).sum())
        named = int((after - keep // case["page"]).sum())
        return {"bytes": 20 * case["n_seq"] + 8 * t + 8 * moved + 4 * named, "flops": 4 * t}
    size, hd = DTYPES[case["dtype"]].itemsize, case["hd"]
    if case["op"] == "append":
        values = t * (case["n_q"] + 2 * case["n_kv"]) * hd
        return {"bytes": values * (size + DTYPES[case["given"]].itemsize) + 8 * t, "flops": 3 * values}
    window = case["window"] or 1 << 40
    rows = int(np.minimum(total, fresh + window - 1).sum())  # cached rows that some new token sees
    pairs = int(sum(np.minimum(np.arange(a, b) + 1, window).sum() for a, b in zip(keep, total)))
    return {"bytes": 2 * rows * case["n_kv"] * hd * size + 2 * t * case["n_q"] * hd * size + 4 * -(-rows // case["page"]),
            "flops": 4 * pairs * case["n_q"] * hd}


def _exact_turn(x, positions, case):
    """The rotation as a complex product in 64 bits."""
    f, factor = _frequencies(case)
    n = f.numel()
    unit = torch.polar(torch.full((len(positions), n), factor, dtype=torch.float64), positions.double().cpu()[:, None] * f).to(x.device)[:, None]
    out = x.double().clone()
    if case["layout"] == "interleaved":
        z = torch.view_as_complex(out[..., : 2 * n].reshape(*out.shape[:-1], n, 2).contiguous()) * unit
        out[..., : 2 * n] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(out[..., :n], out[..., n: 2 * n]) * unit
        out[..., :n], out[..., n: 2 * n] = z.real, z.imag
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_exact_turn(x, s["positions"], case) for x in (s["q"], s["k"]))
    if case["op"] == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        p = case["page"]
        flat_k, flat_v = k.transpose(1, 2).reshape(-1, case["n_kv"], case["hd"]), v.transpose(1, 2).reshape(-1, case["n_kv"], case["hd"])
        flat_k[s["slots"].long()] = _exact_turn(s["k"], s["positions"], case)
        flat_v[s["slots"].long()] = s["v"].double()
        back = lambda x: x.reshape(-1, p, case["n_kv"], case["hd"]).transpose(1, 2)  # noqa: E731
        return {"q": _exact_turn(s["q"], s["positions"], case), "k_pages": back(flat_k), "v_pages": back(flat_v)}
    held, _, fresh = _lengths(case)
    group = case["n_q"] // case["n_kv"]
    out = torch.empty(s["tokens"], case["n_q"], case["hd"], dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["n_seq"]):
        n, total = int(fresh[b]), int(held[b] + fresh[b])
        pages = s["table"][b, : -(-total // case["page"])].long()
        pos = torch.arange(total - n, total, device="cuda")[:, None]
        at = torch.arange(total, device="cuda")[None, :]
        hidden = (at > pos) | ((at <= pos - case["window"]) if case["window"] else (at < 0))
        for h in range(case["n_kv"]):
            k = s["k_pages"][pages, h].reshape(-1, case["hd"])[:total].double()
            v = s["v_pages"][pages, h].reshape(-1, case["hd"])[:total].double()
            for j in range(h * group, (h + 1) * group):
                w = (s["q"][t0:t0 + n, j].double() @ k.T) / math.sqrt(case["hd"])
                if case["softcap"]:
                    w = case["softcap"] * torch.tanh(w / case["softcap"])
                w = w.masked_fill(hidden, -math.inf)
                if s["sink"] is not None:
                    w = torch.cat([w, s["sink"][j].double().expand(n, 1)], 1)
                w = torch.softmax(w, -1)[:, :total]
                out[t0:t0 + n, j] = w @ v
        t0 += n
    return out
