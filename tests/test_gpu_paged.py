"""Paged serving on the GPU against plain references in 64 bits.

Tolerances, from the arithmetic:
- rotation: cos and sin carry the angle's rounding (its top 32 bits become an
  f32 multiple of pi: pi * 2^-25) and sincospi's own error (2^-23 at most), the
  factor one rounding, the two products and their sum 2^-24 each; 16 * 2^-24 of
  (|a| + |b|) * factor covers them.  The result is rounded once: half a step of
  its type (finfo.eps / 2 of the value, half the smallest subnormal below).
- attention: with A = sum_p w_p |v_p| of the reference softmax w, a weight
  rounded to the type moves the output by eps / 2 * A at most (f16 weights below
  the normal range, scaled by 2^8: 2^-33 each, of a sum >= 1); a score summed in
  f32 over hd products is off by hd * 2^-24 * scale * sum |q k| =: d, the softcap
  adds 2^-20 of its bound, so weights are off by 2 d relatively, ex2 and the
  sums by 2^-20; the output is rounded once, eps / 2 of it.
Whole numbers (tables, slots, positions, lengths) are equal.
"""

import ctypes as C
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import kv_cache_decode_attention_gb300 as kvd
    from kv_cache_decode_attention_gb300.build import build

    build()
    return torch, kvd


def _dt(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _tiny(torch, dt):
    return float(torch.finfo(dt).smallest_normal) * float(torch.finfo(dt).eps) / 2


# ---------------------------------------------------------------- rotation

FACTOR = dict(none={}, linear=dict(factor=4.0), ntk=dict(factor=4.0), yarn=dict(factor=8.0, original_len=4096.0),
              bands=dict(factor=8.0, original_len=8192.0))


def _freqs(rot, scaling):
    i = np.arange(0, rot, 2, dtype=np.float64)
    base = 10000.0 * (4.0 ** (rot / (rot - 2)) if scaling == "ntk" else 1.0)
    f, mul = base ** (-i / rot), 1.0
    if scaling == "linear":
        f = f / 4
    if scaling == "yarn":
        dim = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rot - 1)
        r = np.clip((i / 2 - low) / max(high - low, 1e-3), 0, 1)
        f, mul = f / 8 * r + f * (1 - r), 0.1 * math.log(8) + 1
    if scaling == "bands":
        m = np.clip((8192 * f / (2 * math.pi) - 1) / 3, 0, 1)
        f = f / 8 * (1 - m) + f * m
    return f, mul


def _turn(x, pos, rot, layout, scaling):
    """x [t, h, hd] f64 turned, and |a| + |b| of each channel's pair (0 past rot)."""
    f, mul = _freqs(rot, scaling)
    # the angle's turns in exact integers: positions up to 2^31 times a 64-bit fraction
    frac = [[(int(p) * round(fi / (2 * math.pi) * 2 ** 64)) % 2 ** 64 / 2 ** 64 for fi in f] for p in pos]
    a = np.array(frac)[:, None, :] * 2 * math.pi
    c, s = np.cos(a) * mul, np.sin(a) * mul
    n = rot // 2
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if layout == "interleaved" else (slice(0, n), slice(n, rot))
    out, size = x.copy(), np.zeros_like(x)
    out[..., one], out[..., two] = x[..., one] * c - x[..., two] * s, x[..., two] * c + x[..., one] * s
    size[..., one] = size[..., two] = (np.abs(x[..., one]) + np.abs(x[..., two])) * mul
    return out, size


def _check_turn(torch, got, want, size, dt):
    tol = 16 * 2 ** -24 * size + float(torch.finfo(dt).eps) / 2 * (np.abs(want) + 16 * 2 ** -24 * size) + _tiny(torch, dt)
    d = np.abs(got.double().cpu().numpy() - want)
    assert (d <= tol).all(), (float((d - tol).max()), np.unravel_index((d - tol).argmax(), d.shape))


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("hd,rot,dtype", [(128, 128, "bf16"), (64, 64, "f16"), (128, 64, "f32"), (128, 70, "bf16"), (64, 32, "f32"), (80, 48, "f16"),
                                          (33, 2, "f32"), (512, 512, "bf16"), (256, 16, "f16"), (7, 6, "bf16")])
def test_rope_sizes(env, layout, hd, rot, dtype):
    torch, kvd = env
    dt = _dt(torch, dtype)
    g = torch.Generator(device="cuda").manual_seed(hd * 1000 + rot)
    for t, n_q, n_kv in ((1, 8, 2), (5, 3, 3), (700, 4, 1)):
        q = torch.randn(t, n_q, hd, generator=g, device="cuda").to(dt)
        k = torch.randn(t, n_kv, hd, generator=g, device="cuda").to(dt)
        pos = torch.randint(0, 1 << 20, (t,), generator=g, device="cuda", dtype=torch.int32)
        qo, ko = kvd.rope(q, k, pos, kvd.RopeTable(rot, layout))
        for x, o in ((q, qo), (k, ko)):
            want, size = _turn(x.double().cpu().numpy(), pos.tolist(), rot, layout, "none")
            _check_turn(torch, o, want, size, dt)
            assert torch.equal(o[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
def test_rope_scalings_and_far_positions(env, scaling):
    torch, kvd = env
    pos = [0, 1, 2, 4095, 4096, 131071, 10 ** 6 + 1, 2 ** 31 - 1]
    x = torch.randn(len(pos), 3, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    o, none = kvd.rope(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), kvd.RopeTable(128, "half", scaling, **FACTOR[scaling]))
    assert none is None
    # at 2^31 the f64 rounding of f itself (2^-53 * f, a few of them) moves the angle by 2^31 * f * 2^-50
    want, size = _turn(x.double().cpu().numpy(), pos, 128, "half", scaling)
    _check_turn(torch, o, want, size + np.array(pos, np.float64)[:, None, None] * 2.0 ** -50 / (16 * 2 ** -24) * size, torch.float32)


def test_rope_slices_in_place_and_padding(env):
    """q and k as slices of one projection, in place, and rows without a position."""
    torch, kvd = env
    g = torch.Generator(device="cuda").manual_seed(3)
    for hd, rot in ((128, 128), (128, 70), (64, 16)):
        qkv = torch.randn(9, 14, hd, generator=g, device="cuda").to(torch.bfloat16)
        pos = torch.tensor([5, -1, 7, 8, -1, -2, 3, 3, 0], dtype=torch.int32, device="cuda")
        table = kvd.RopeTable(rot)
        apart = kvd.rope(qkv[:, :8], qkv[:, 8:11], pos, table, q_out=torch.full((9, 8, hd), 7.0, device="cuda", dtype=torch.bfloat16),
                         k_out=torch.full((9, 3, hd), 7.0, device="cuda", dtype=torch.bfloat16))
        before = qkv.clone()
        q, k = qkv[:, :8], qkv[:, 8:11]
        kvd.rope(q, k, pos, table, q_out=q, k_out=k)
        skip = (pos < 0).cpu()
        for a, b, old in ((apart[0], q, before[:, :8]), (apart[1], k, before[:, 8:11])):
            assert torch.equal(a[~skip], b[~skip]) and torch.equal(b[skip], old[skip]) and bool((a[skip] == 7).all())
            want, size = _turn(old.double().cpu().numpy(), [max(p, 0) for p in pos.tolist()], rot, "half", "none")
            keep = (~skip).numpy()
            _check_turn(torch, a[~skip], want[keep], size[keep], torch.bfloat16)
        assert torch.equal(qkv[:, 11:], before[:, 11:])
        odd = torch.randn(9, 5, hd + 1, generator=g, device="cuda").to(torch.bfloat16)[..., 1:]  # rows that 16-byte accesses cannot take
        want, size = _turn(odd.double().cpu().numpy(), [max(p, 0) for p in pos.tolist()], rot, "half", "none")
        _check_turn(torch, kvd.rope(None, odd, pos, table)[1][~skip], want[keep], size[keep], torch.bfloat16)
    empty = kvd.rope(torch.empty(0, 4, 64, device="cuda"), None, torch.empty(0, dtype=torch.int32, device="cuda"), kvd.RopeTable(64))[0]
    assert empty.shape == (0, 4, 64)


def test_rotated_rows_feed_the_contiguous_cache(env):
    """rope's f32 rows go into kv_append and decode_attention: scores depend on the
    distance alone, so a shift of all positions leaves the output as it is."""
    torch, kvd = env
    g = torch.Generator(device="cuda").manual_seed(5)
    L, n_kv, hd = 40, 2, 64
    k, v = torch.randn(L, n_kv, hd, generator=g, device="cuda"), torch.randn(L, n_kv, hd, generator=g, device="cuda")
    q = torch.randn(1, 4, hd, generator=g, device="cuda")
    outs = []
    for shift in (0, 7777):
        table = kvd.RopeTable(hd, "interleaved")
        kr = kvd.rope(None, k, torch.arange(shift, shift + L, device="cuda", dtype=torch.int32), table)[1]
        qr = kvd.rope(q, None, torch.tensor([shift + L - 1], device="cuda", dtype=torch.int32), table)[0]
        layer = kvd.LayerKvCache(1, n_kv, hd, "f32", L)
        kvd.kv_append(layer, kr, v, [L])
        outs.append(kvd.decode_attention(qr.contiguous(), layer))
    # scores: hd products of rows off by 16 * 2^-24 (|a| + |b|) each, |x| < 6
    assert float((outs[0] - outs[1]).abs().max()) <= 2 * hd * 2 * 16 * 2 ** -24 * 2 * 36 / math.sqrt(hd) * 6


# ---------------------------------------------------------------- plan


class Model:
    """The plan, step by step on Python lists."""

    def __init__(self, n_seq, page, width, n_pages):
        self.page, self.width = page, width
        self.len, self.pages, self.free = [0] * n_seq, [[] for _ in range(n_seq)], list(range(n_pages - 1, -1, -1))

    def step(self, new, keep, room):
        keep = list(self.len) if keep is None else keep
        after = [-(-(a + b) // self.page) for a, b in zip(keep, new)]
        gone = [p[n:] for p, n in zip(self.pages, after)]
        need = sum(max(0, n - len(p)) for p, n in zip(self.pages, after))
        if max(after) > self.width or need > len(self.free) + sum(map(len, gone)) or sum(new) > room:
            return None
        self.free += [x for g in gone for x in g]
        for b, n in enumerate(after):
            self.pages[b] = self.pages[b][:n]
            while len(self.pages[b]) < n:
                self.pages[b].append(self.free.pop())
        pos = [[k + i for i in range(n)] for k, n in zip(keep, new)]
        slots = [[self.pages[b][p // self.page] * self.page + p % self.page for p in ps] for b, ps in enumerate(pos)]
        self.len = [a + b for a, b in zip(keep, new)]
        return [sum(new[:b]) for b in range(len(new) + 1)], sum(pos, []), sum(slots, [])


def _i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same_state(cache, model):
    assert cache.seq_len.tolist() == model.len
    n = int(cache.n_free)
    assert cache.free_pages[:n].tolist() == model.free
    table = cache.block_table.cpu().numpy()
    for b, p in enumerate(model.pages):
        assert table[b, : len(p)].tolist() == p, b


@pytest.mark.parametrize("n_seq,page,width,n_pages,most", [(1, 16, 8, 8, 60), (7, 16, 10, 40, 40), (33, 32, 6, 120, 90), (1500, 16, 3, 3000, 20), (1500, 16, 12, 12000, 20), (5, 128, 50, 200, 2500),
                                                            (8192, 16, 4, 20000, 12)])
def test_plan_follows_a_simple_allocator(env, n_seq, page, width, n_pages, most):
    torch, kvd = env
    r = np.random.default_rng(n_seq)
    cache = kvd.PagedKvCache(n_pages, page, 1, 64, n_seq, width)
    model = Model(n_seq, page, width, n_pages)
    steps = refused = 0
    for step in range(12):
        new = r.integers(0, most, n_seq) * (r.random(n_seq) < 0.7)
        keep = None if step % 3 == 0 else [int(r.integers(0, n + 1)) if r.random() < 0.3 else n for n in model.len]
        if step % 4 == 3:
            keep = [0 if r.random() < 0.6 else n for n in model.len]
        room = int(new.sum()) + int(r.integers(0, 50))
        old = cache.seq_len.clone(), cache.n_free.clone(), cache.block_table.clone(), list(model.free), [list(p) for p in model.pages]
        want = model.step(new.tolist(), keep, room)
        keep_t = None if keep is None else _i32(torch, keep)
        if step % 2:  # planned apart first: the same answer, the state unmoved, and again in place
            apart = kvd.paged_plan(cache, _i32(torch, new.tolist()), room, keep_len=keep_t, advance=False)
            assert torch.equal(cache.seq_len, old[0]) and torch.equal(cache.n_free, old[1])
            cache.device_error()
        plan = kvd.paged_plan(cache, _i32(torch, new.tolist()), room, keep_len=keep_t)
        if want is None:
            refused += 1
            assert cache.device_error() == 4
            assert torch.equal(cache.seq_len, old[0]) and torch.equal(cache.n_free, old[1]) and torch.equal(cache.block_table, old[2])
            assert not plan.cu_new.any() and bool((plan.slots == -1).all()) and bool((plan.positions == -1).all())
        else:
            steps += 1
            cu, pos, slots = want
            pad = [-1] * (room - cu[-1])
            assert plan.cu_new.tolist() == cu and plan.positions.tolist() == pos + pad and plan.slots.tolist() == slots + pad
            assert cache.device_error() == 0
        if step % 2:
            for x, y in ((apart.cu_new, plan.cu_new), (apart.positions, plan.positions), (apart.slots, plan.slots), (apart.seq_len, cache.seq_len), (apart.n_free, cache.n_free)):
                assert torch.equal(x, y)
        _same_state(cache, model)
    assert steps >= 2 and steps + refused == 12


def test_plan_fills_buffers_at_any_offset(env):
    """Rows in runs of four where the buffers allow it, one by one where they do not: the same plan."""
    torch, kvd = env
    cache = kvd.PagedKvCache(2000, 16, 1, 64, 7, 800)
    new = _i32(torch, [9001, 3, 0, 1200, 5, 0, 4000])
    room = 14221
    want = kvd.paged_plan(cache, new, room, advance=False)
    for off in (0, 1, 2, 3):
        pos, slots = (torch.full((room + 8,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        plan = kvd.PagedPlan(torch.empty_like(want.cu_new), torch.empty_like(want.seq_len), torch.empty_like(want.n_free), pos[off:off + room], slots[off:off + room])
        kvd.paged_plan(cache, new, room, advance=False, plan=plan)
        assert torch.equal(plan.positions, want.positions) and torch.equal(plan.slots, want.slots)
        for x in (pos, slots):
            assert bool((x[:off] == 77).all()) and bool((x[off + room:] == 77).all())
    assert cache.device_error() == 0


def test_plan_refuses_what_does_not_fit_or_is_malformed(env):
    torch, kvd = env
    cache = kvd.PagedKvCache(6, 16, 1, 64, 3, 4)
    kvd.paged_plan(cache, _i32(torch, [20, 0, 33]), 53)  # 2 + 0 + 3 pages of 6
    state = [t.clone() for t in (cache.seq_len, cache.n_free, cache.block_table, cache.free_pages)]
    for new, keep, room, bit in (([0, 30, 0], None, 100, 4),        # two pages, one is free
                                 ([0, 0, 40], None, 100, 4),        # 73 rows in a table of 4 pages
                                 ([1, 1, 1], None, 2, 4),           # room for two rows
                                 ([-1, 0, 0], None, 100, 2), ([0, 0, 0], [21, 0, 0], 100, 2), ([0, 0, 0], [20, -1, 33], 100, 2),
                                 ([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1], None, 100, 4)):
        plan = kvd.paged_plan(cache, _i32(torch, new), room, keep_len=None if keep is None else _i32(torch, keep))
        assert cache.device_error() == bit, (new, keep)
        assert not plan.cu_new.any() and bool((plan.slots == -1).all())
        for a, b in zip(state[:3], (cache.seq_len, cache.n_free, cache.block_table)):
            assert torch.equal(a, b)
    # dropping one request makes the room another needs, in one step
    kvd.paged_plan(cache, _i32(torch, [0, 60, 0]), 60, keep_len=_i32(torch, [20, 0, 0]))
    assert cache.device_error() == 0 and cache.seq_len.tolist() == [20, 60, 0] and int(cache.n_free) == 0
    assert sorted(cache.block_table[0, :2].tolist() + cache.block_table[1, :4].tolist()) == list(range(6))
    # a step of no rows at all
    plan = kvd.paged_plan(cache, _i32(torch, [0, 0, 0]), 0)
    assert cache.device_error() == 0 and plan.cu_new.tolist() == [0, 0, 0, 0] and plan.slots.numel() == 0


# ---------------------------------------------------------------- append


@pytest.mark.parametrize("given,pages", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("hd,rot,layout", [(128, 128, "half"), (64, 32, "interleaved"), (128, 38, "half"), (64, 0, "")])
def test_append_rotates_and_places_rows(env, given, pages, hd, rot, layout):
    torch, kvd = env
    gi, gp = _dt(torch, given), _dt(torch, pages)
    n_kv, n_q, page = 3, 6, 32
    g = torch.Generator(device="cuda").manual_seed(hd + rot)
    cache = kvd.PagedKvCache(20, page, n_kv, hd, 4, 10, dtype=gp)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    plan = kvd.paged_plan(cache, _i32(torch, [50, 0, 1, 97]), 160)  # 148 rows, 12 places behind them
    qkv = torch.randn(160, n_q + 2 * n_kv, hd, generator=g, device="cuda").to(gi)
    q, k, v = qkv[:, :n_q], qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    q_out = torch.full((160, n_q, hd), 3.0, device="cuda", dtype=gp)
    table = kvd.RopeTable(rot, layout) if rot else None
    assert kvd.paged_append(cache, plan, k, v, q=q, q_out=q_out, rope=table) is q_out
    assert cache.device_error() == 0
    pos, slots = plan.positions[:148].tolist(), plan.slots[:148].cpu()
    assert bool((q_out[148:] == 3).all())
    for x, o in ((q[:148], q_out[:148]), (k[:148], cache.k.transpose(1, 2).reshape(-1, n_kv, hd)[slots.long().cuda()])):
        x64 = x.double().cpu().numpy()
        want, size = _turn(x64, pos, rot, layout, "none") if rot else (x64, np.zeros_like(x64))
        _check_turn(torch, o, want, size, gp)
    assert torch.equal(cache.v.transpose(1, 2).reshape(-1, n_kv, hd)[slots.long().cuda()], v[:148].to(gp))
    held = torch.zeros(20 * page, dtype=torch.bool)
    held[slots.long()] = True
    for t in (cache.k, cache.v):  # nothing else was touched
        assert bool(torch.isnan(t.transpose(1, 2).reshape(20 * page, -1)[~held.cuda()]).all())


def test_append_in_place_captured_and_with_a_slot_twice(env):
    torch, kvd = env
    g = torch.Generator(device="cuda").manual_seed(3)
    cache, other = kvd.PagedKvCache(8, 16, 2, 64, 2, 4), kvd.PagedKvCache(8, 16, 2, 64, 2, 4)
    plan = kvd.paged_plan(cache, _i32(torch, [20, 9]), 33)
    x = torch.randn(33, 10, 64, device="cuda", generator=g).bfloat16()
    table = kvd.RopeTable(64, "half")
    for c in (cache, other):
        c.k.zero_()
        c.v.zero_()
    want = kvd.paged_append(cache, plan, x[:, 6:8], x[:, 8:], q=x[:, :6], rope=table)
    y = x.clone()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert kvd.paged_append(other, plan, y[:, 6:8], y[:, 8:], q=y[:, :6], q_out=y[:, :6], rope=table).data_ptr() == y.data_ptr()
    for _ in range(2):
        y.copy_(x)
        graph.replay()
        assert torch.equal(y[:29, :6], want[:29]) and torch.equal(y[29:], x[29:]) and torch.equal(y[:, 6:], x[:, 6:])
        assert torch.equal(other.k, cache.k) and torch.equal(other.v, cache.v)
    twice = kvd.PagedPlan(None, None, positions=_i32(torch, [0, 1]), slots=_i32(torch, [5, 5]))
    kvd.paged_append(other, twice, x[:2, 6:8], x[:2, 8:])
    got = other.v.transpose(1, 2).reshape(-1, 2, 64)[5]
    assert bool(((got == x[0, 8:]) | (got == x[1, 8:])).all())
    assert other.device_error() == 0 and cache.device_error() == 0


def test_append_skips_bad_slots(env):
    torch, kvd = env
    cache = kvd.PagedKvCache(2, 16, 2, 64, 1, 2)
    cache.k.zero_()
    cache.v.zero_()
    x = torch.ones(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    plan = kvd.PagedPlan(None, None, positions=_i32(torch, [0, 1, 2, 3]), slots=_i32(torch, [31, 32, -5, 2 ** 31 - 1]))
    assert kvd.paged_append(cache, plan, x, x) is None
    assert cache.device_error() == 2 and cache.device_error() == 0
    assert int((cache.v != 0).sum()) == 2 * 64 and bool((cache.v[1, :, 15] == 1).all()) and bool((cache.k[1, :, 15] == 1).all())
    none = kvd.PagedPlan(None, None, positions=_i32(torch, []), slots=_i32(torch, []))
    kvd.paged_append(cache, none, x[:0], x[:0])


# ---------------------------------------------------------------- attention


def _attend(torch, q, k, v, total, scale, window=0, softcap=0.0, sink=None):
    """64-bit attention of q [n, n_q, hd], the last n of `total` rows k, v [total, n_kv, hd]; returns out and its tolerance but for the
    type's rounding: (out, A, slack) with slack the relative error of the weights."""
    n, n_q, hd = q.shape
    grp = n_q // k.shape[1]
    pos = torch.arange(total - n, total, device=q.device)[:, None]
    at = torch.arange(total, device=q.device)[None, :]
    seen = at <= pos
    if window:
        seen &= at > pos - window
    out = torch.zeros(n, n_q, hd, dtype=torch.float64, device=q.device)
    size, slack = torch.zeros_like(out), torch.zeros(n, n_q, 1, dtype=torch.float64, device=q.device)
    for h in range(n_q):
        x, kk, vv = q[:, h].double(), k[:, h // grp].double(), v[:, h // grp].double()
        s = x @ kk.T * scale
        d = hd * 2.0 ** -24 * scale * (x.abs() @ kk.abs().T)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            d = d + 2.0 ** -20 * softcap
        s = s.masked_fill(~seen, -math.inf)
        top = s.max(-1, keepdim=True).values if total else torch.full((n, 1), -math.inf, dtype=torch.float64, device=q.device)
        if sink is not None:
            top = torch.maximum(top, sink[h].double())
        w = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
        below = w.sum(-1, keepdim=True) + (torch.exp(sink[h].double() - top) if sink is not None else 0)
        w = torch.where(seen.any(-1, keepdim=True), w / below, torch.zeros_like(w))
        out[:, h], size[:, h] = w @ vv, w @ vv.abs()
        slack[:, h] = 2 * (d * seen).max(-1, keepdim=True).values if total else 0
    return out, size, slack + 2.0 ** -20


def _check_attend(torch, got, want, size, slack, dt, vmax):
    half = float(torch.finfo(dt).eps) / 2
    # the weights' rounding, the scores' error, f16 weights below the normal range, and the output's rounding
    tol = (half + slack * (1 + half)) * size * (1 + half) + half * want.abs() + _tiny(torch, dt) + (0 if dt == torch.bfloat16 else 2.0 ** -33 * 2 ** 17 * vmax)
    d = (got.double() - want).abs()
    assert not bool(torch.isnan(got).any())
    assert bool((d <= tol).all()), float((d / tol).max())


def _poisoned(torch, kvd, lens, n_kv, hd, page, dt, seed, spare=3):
    """Pages of random rows for requests of these lengths, shuffled, with NaN in every row that no request holds and nonsense in the
    table's unused places; the rows of each request beside it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    has = [-(-n // page) for n in lens]
    n_pages = sum(has) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    width = max(has) + 2
    k = torch.full((n_pages, n_kv, page, hd), float("nan"), device="cuda", dtype=dt)
    v = torch.full_like(k, float("nan"))
    table = torch.tensor([[2 ** 31 - 1, -7, n_pages][i % 3] for i in range(len(lens) * width)], dtype=torch.int32).view(len(lens), width)
    rows = []
    for b, n in enumerate(lens):
        kk = torch.randn(n, n_kv, hd, generator=g, device="cuda").to(dt)
        vv = torch.randn(n, n_kv, hd, generator=g, device="cuda").to(dt)
        rows.append((kk, vv))
        for i in range(has[b]):
            p = order.pop()
            table[b, i] = p
            part = slice(i * page, min(n, (i + 1) * page))
            k[p, :, : part.stop - part.start] = kk[part].transpose(0, 1)
            v[p, :, : part.stop - part.start] = vv[part].transpose(0, 1)
    return kvd.PagedKvCache.of(k, v, table.cuda(), _i32(torch, lens)), rows


def _run_attend(torch, kvd, lens, new, n_kv, group, hd, page, dt, seed, window=0, softcap=0.0, sinks=False, scale=None, tail=3, sample=None):
    cache, rows = _poisoned(torch, kvd, lens, n_kv, hd, page, dt, seed)
    t = sum(new)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = (torch.randn(t + tail, n_kv * group, hd, generator=g, device="cuda") * 1.5).to(dt)
    q[t:] = float("nan")
    sink = torch.randn(n_kv * group, generator=g, device="cuda") * 2 if sinks else None
    plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
    out = torch.full_like(q, 9.0)
    scale = 1 / math.sqrt(hd) if scale is None else scale
    assert kvd.paged_attention(q, cache, plan, out=out, scale=scale, window=window, softcap=softcap, sinks=sink) is out
    assert cache.device_error() == 0
    assert bool((out[t:] == 9).all())
    at = 0
    for b, n in enumerate(new):
        if n and (sample is None or b in sample):
            kk, vv = rows[b]
            live = min(n, lens[b])  # a position below zero sees nothing
            assert not out[at:at + n - live].any()
            if live:
                want = _attend(torch, q[at + n - live:at + n], kk, vv, lens[b], scale, window, softcap, sink)
                _check_attend(torch, out[at + n - live:at + n], *want, dt, float(vv.abs().max()))
        at += n
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,page", [(1, 16), (4, 64), (16, 128), (5, 32)])
def test_attention_of_single_tokens(env, dtype, hd, group, page):
    torch, kvd = env
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700, 0, 2049]
    _run_attend(torch, kvd, lens, [1 if n else 0 for n in lens], 2, group, hd, page, _dt(torch, dtype), group)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,page", [(1, 128), (2, 16), (3, 32), (8, 64), (16, 16)])
def test_attention_of_chunks(env, dtype, hd, group, page):
    """Chunks around the tile's edges: one tile, one row over, two tiles and over."""
    torch, kvd = env
    tile = 128 // group
    new = [1, tile - 1 or 1, tile, tile + 1, 2 * tile, 2 * tile + 1, 0, 4 * tile + 3, 3 * tile, 7]
    lens = [n + x for n, x in zip(new, [0, 5, 128 - tile if tile < 128 else 0, 300, 0, 77, 9, 1000, 129, 1500])]
    _run_attend(torch, kvd, lens, new, 2, group, hd, page, _dt(torch, dtype), 100 + group)


@pytest.mark.parametrize("hd,group", [(64, 2), (128, 4), (128, 1)])
@pytest.mark.parametrize("window,softcap,sinks", [(1, 0.0, False), (2, 0.0, True), (100, 0.0, False), (128, 30.0, False), (1000, 5.0, True), (0, 30.0, False),
                                                  (0, 0.0, True), (1 << 40, 0.0, False)])
def test_attention_options(env, hd, group, window, softcap, sinks):
    torch, kvd = env
    for dt in (torch.bfloat16, torch.float16):
        _run_attend(torch, kvd, [900, 1, 130, 2000, 64], [1, 1, 130, 300, 3], 2, group, hd, 16, dt, 7, window, softcap, sinks)


def test_attention_rows_that_see_nothing_are_zero(env):
    """More new rows than rows held: the first ones stand before the start."""
    torch, kvd = env
    for sinks in (False, True):
        _run_attend(torch, kvd, [3, 0, 130, 0], [5, 2, 400, 1], 2, 4, 128, 16, torch.bfloat16, 11, sinks=sinks)


def test_attention_cuts_long_requests(env):
    """One long request among short ones, and one alone: items cut over many CTAs and joined, with and without options."""
    torch, kvd = env
    for dt, hd in ((torch.bfloat16, 128), (torch.float16, 64)):
        _run_attend(torch, kvd, [60001], [1], 1, 8, hd, 64, dt, 21)
        _run_attend(torch, kvd, [30011, 5, 900], [3, 5, 1], 2, 4, hd, 16, dt, 22, sinks=True)
        _run_attend(torch, kvd, [9000], [700], 1, 4, hd, 128, dt, 23, softcap=20.0, sinks=True)
        _run_attend(torch, kvd, [20000], [130], 1, 1, hd, 32, dt, 24, window=5000)


def test_attention_of_many_requests(env):
    """More requests than threads plan the cut with: some empty, most short."""
    torch, kvd = env
    r = np.random.default_rng(2)
    lens = r.integers(0, 40, 1100).tolist()
    new = [int(r.integers(0, min(n, 3) + 1)) for n in lens]
    _run_attend(torch, kvd, lens, new, 1, 2, 64, 16, torch.bfloat16, 31, sample=set(range(0, 1100, 13)) | {0, 1, 1098, 1099})
    none = _run_attend(torch, kvd, [5, 7], [0, 0], 1, 2, 64, 16, torch.bfloat16, 31)
    assert none.shape[0] == 3


@pytest.mark.parametrize("seed", range(12))
def test_attention_of_mixed_batches(env, seed):
    """Prompts, drafts, single tokens, requests without new rows and without rows, in any order and length: items of two query tiles and
    of one, whole and cut, with and without a short last page, follow one another in a CTA."""
    torch, kvd = env
    r = np.random.default_rng(900 + seed)
    hd, dt = (64, 128)[seed % 2], (torch.bfloat16, torch.float16)[seed // 2 % 2]
    group, page, n_kv = int(r.choice([1, 2, 4, 8])), int(r.choice([16, 32, 64, 128])), int(r.choice([1, 3, 8]))
    lens, new = [], []
    for _ in range(int(r.integers(20, 120))):
        kind = r.random()
        n = 1 if kind < 0.4 else int(r.integers(2, 9)) if kind < 0.6 else int(r.integers(9, 400)) if kind < 0.85 else 0
        past = int(r.integers(0, 300)) if r.random() < 0.6 else int(r.integers(0, 3000))
        new.append(n)
        lens.append(n + past)
    sample = set(r.choice(len(lens), 25).tolist())
    _run_attend(torch, kvd, lens, new, n_kv, group, hd, page, dt, 900 + seed, window=int(r.choice([0, 0, 200])), softcap=float(r.choice([0.0, 0.0, 20.0])),
                sinks=bool(r.random() < 0.3), sample=sample)


def test_attention_over_many_batches(env):
    """Hundreds of drawn batches, each computed three times beside copies on another stream: the same bits, no wait that gave up, no row
    left out, and one request of each against 64 bits."""
    torch, kvd = env
    r = np.random.default_rng(77)
    side = torch.cuda.Stream()
    src, dst = (torch.zeros(1 << 26, device="cuda", dtype=torch.uint8) for _ in range(2))
    for i in range(400):
        hd, page, dt = int(r.choice([64, 64, 128])), int(r.choice([16, 32, 64, 128])), (torch.bfloat16, torch.float16)[i % 2]
        n_kv, group, n_seq = int(r.choice([1, 2, 8])), int(r.choice([1, 2, 4, 5, 8, 16])), int(2 ** r.uniform(0, 9))
        kind, room = r.random(n_seq), 2 ** r.uniform(3, 12)
        new = np.where(kind < 0.5, 1, np.where(kind < 0.7, r.integers(0, 9, n_seq), (2 ** r.uniform(3, 9, n_seq)).astype(int)))
        lens = new + (r.random(n_seq) * room).astype(int)
        has = -(-lens // page)
        table = np.full((n_seq, has.max() + 1), -1, dtype=np.int32)
        order, at = r.permutation(int(has.sum()) + 1).astype(np.int32), 0
        for b in range(n_seq):
            table[b, : has[b]] = order[at:at + has[b]]
            at += has[b]
        k, v = (torch.randn(len(order), n_kv, page, hd, device="cuda").to(dt) for _ in range(2))
        cache = kvd.PagedKvCache.of(k, v, torch.from_numpy(table).cuda(), _i32(torch, lens.tolist()))
        cu = np.concatenate([[0], np.cumsum(new)])
        plan = kvd.PagedPlan(_i32(torch, cu.tolist()), cache.seq_len)
        q = torch.randn(int(cu[-1]), n_kv * group, hd, device="cuda").to(dt)
        window, cap = int(r.choice([0, 0, 100, 1000])), float(r.choice([0.0, 0.0, 20.0]))
        outs = []
        for _ in range(3):
            with torch.cuda.stream(side):
                dst.copy_(src)
            outs.append(kvd.paged_attention(q, cache, plan, out=torch.full_like(q, float("nan")), window=window, softcap=cap))
        assert cache.device_error() == 0, i
        assert not bool(torch.isnan(outs[0]).any()) and all(torch.equal(outs[0], x) for x in outs), i
        b = int(r.integers(n_seq))
        if new[b] and new[b] * lens[b] * n_kv * group < 1 << 22:
            kk, vv = (x[cache.block_table[b, : has[b]].long()].transpose(1, 2).reshape(-1, n_kv, hd)[: lens[b]] for x in (k, v))
            part = slice(int(cu[b]), int(cu[b + 1]))
            _check_attend(torch, outs[0][part], *_attend(torch, q[part], kk, vv, int(lens[b]), hd ** -0.5, window, cap), dt, float(vv.abs().max()))


def test_requests_may_share_pages_and_rows_may_be_broadcast(env):
    """A common beginning held once; one query row for all tokens or heads (strides of zero)."""
    torch, kvd = env
    cache, rows = _poisoned(torch, kvd, [700, 700], 2, 128, 32, torch.bfloat16, 5)
    cache.block_table[1, :20] = cache.block_table[0, :20]  # rows 0 .. 639
    k1, v1 = (torch.cat([a[:640], b[640:]]) for a, b in zip(rows[0], rows[1]))
    q = torch.randn(1, 1, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    plan = kvd.PagedPlan(_i32(torch, [0, 30, 60]), cache.seq_len)
    for wide in (q.expand(60, 8, 128), q.expand(60, 1, 128).contiguous().expand(60, 8, 128), q.expand(1, 8, 128).contiguous().expand(60, 8, 128)):
        out = kvd.paged_attention(wide, cache, plan)
        assert out.is_contiguous() and torch.equal(out, kvd.paged_attention(wide.contiguous(), cache, plan))
        for at, (k, v) in ((0, rows[0]), (30, (k1, v1))):
            _check_attend(torch, out[at:at + 30], *_attend(torch, wide[at:at + 30], k, v, 700, 128 ** -0.5), torch.bfloat16, float(v.abs().max()))
    assert cache.device_error() == 0


@pytest.mark.parametrize("scale", [1e-6, 1.0, 20.0])
def test_attention_of_flat_and_sharp_softmaxes(env, scale):
    """From a plain mean of all rows to one row that takes everything, over many tiles: the running maximum moves or stays."""
    torch, kvd = env
    for dt in (torch.bfloat16, torch.float16):
        _run_attend(torch, kvd, [1500, 400], [1, 300], 1, 4, 64, 16, dt, 41, scale=scale)


def test_attention_with_growing_scores(env):
    """Keys that grow with their position make the maximum move at every tile; falling ones never."""
    torch, kvd = env
    for rising in (True, False):
        cache, rows = _poisoned(torch, kvd, [1024], 1, 64, 16, torch.bfloat16, 51)
        f = torch.linspace(0, 6, 1024, device="cuda")
        f = f if rising else f.flip(0)
        q = torch.ones(40, 4, 64, device="cuda", dtype=torch.bfloat16)
        kk = (f[:, None, None] * torch.ones(1, 1, 64, device="cuda")).to(torch.bfloat16)
        cache.k[cache.block_table[0, :64].long()] = kk.view(64, 16, 1, 64).transpose(1, 2)
        plan = kvd.PagedPlan(_i32(torch, [0, 40]), cache.seq_len)
        out = kvd.paged_attention(q, cache, plan)
        _check_attend(torch, out, *_attend(torch, q, kk, rows[0][1], 1024, 1 / 8), torch.bfloat16, 5.0)


def test_attention_takes_views(env):
    """q as a slice of one projection, out as a slice of a wider array."""
    torch, kvd = env
    cache, rows = _poisoned(torch, kvd, [300, 40], 2, 128, 32, torch.float16, 61)
    qkv = torch.randn(150, 12, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).half()
    wide = torch.full((150, 10, 192), 4.0, device="cuda", dtype=torch.float16)
    q, out = qkv[:, 2:10], wide[:, 1:9, 64:]
    plan = kvd.PagedPlan(_i32(torch, [0, 130, 150]), cache.seq_len)
    kvd.paged_attention(q, cache, plan, out=out)
    assert torch.equal(out, kvd.paged_attention(q.contiguous(), cache, plan))
    assert bool((wide[:, 0] == 4).all()) and bool((wide[:, 9] == 4).all()) and bool((wide[..., :64] == 4).all())
    for b, (a, e) in enumerate(((0, 130), (130, 150))):
        _check_attend(torch, out[a:e], *_attend(torch, q[a:e], *rows[b], rows[b][0].shape[0], 128 ** -0.5), torch.float16, 5.0)
    for bad in (qkv[:, 2:10, ::2], torch.empty(150, 8, 129, device="cuda", dtype=torch.float16)[..., 1:]):
        with pytest.raises((ValueError, kvd.KvdError)):
            kvd.paged_attention(bad, cache, plan)


def test_attention_skips_malformed_requests(env):
    """A request whose numbers cannot be, and a page past the pool: the error bit, and every other request as it should be."""
    torch, kvd = env
    lens, new = [100, 60, 70, 300], [2, 1, 4, 1]
    cache, rows = _poisoned(torch, kvd, lens, 1, 64, 16, torch.bfloat16, 71)
    q = torch.randn(8, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).bfloat16()
    cu = [0, 2, 3, 7, 8]
    good = kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, cu), cache.seq_len))
    wide = cache.block_table.shape[1] * 16
    for bad_len in (-1, wide + 1, 2 ** 31 - 1):
        seq = _i32(torch, [100, bad_len, 70, 300])
        out = torch.full_like(q, 5.0)
        kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, cu), seq), out=out)
        assert cache.device_error() == 2
        assert bool((out[2] == 5).all())
        for a, e, b in ((0, 2, 0), (3, 7, 2), (7, 8, 3)):
            _check_attend(torch, out[a:e], *_attend(torch, q[a:e], *rows[b], lens[b], 1 / 8), torch.bfloat16, 5.0)
    for bad_cu in ([0, 2, 1, 7, 8], [0, 2, 3, 7, 9], [-1, 2, 3, 7, 8]):
        out = torch.full_like(q, 5.0)
        kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, bad_cu), cache.seq_len), out=out)
        assert cache.device_error() == 2
    cache.block_table[3, 2] = cache.n_pages
    out = kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, cu), cache.seq_len))
    assert cache.device_error() == 2
    for a, e, b in ((0, 2, 0), (2, 3, 1), (3, 7, 2)):
        _check_attend(torch, out[a:e], *_attend(torch, q[a:e], *rows[b], lens[b], 1 / 8), torch.bfloat16, 5.0)
    assert not bool(torch.isnan(out).any()) and good.shape == out.shape


# ---------------------------------------------------------------- together


class Server:
    """Requests on Python lists beside the cache: what each holds, in the pages' dtype, and its tokens' queries."""

    def __init__(self, torch, kvd, n_seq, n_kv, group, hd, page, n_pages, width, dt, layers=2, window=0):
        self.torch, self.kvd, self.window = torch, kvd, window
        self.caches = [kvd.PagedKvCache(n_pages, page, n_kv, hd, n_seq, width, dtype=dt)]
        self.caches += [self.caches[0].layer_like() for _ in range(layers - 1)]
        for c in self.caches:
            c.k.fill_(float("nan"))
            c.v.fill_(float("nan"))
        self.held = [[torch.empty(0, 2 * n_kv, hd, device="cuda", dtype=dt) for _ in range(n_seq)] for _ in range(layers)]
        self.table = kvd.RopeTable(hd, "half", "yarn", factor=8.0, original_len=256.0)
        self.n_kv, self.n_q, self.hd, self.dt, self.n_seq = n_kv, n_kv * group, hd, dt, n_seq

    def inputs(self, room, seed):
        g = self.torch.Generator(device="cuda").manual_seed(seed)
        return [self.torch.randn(room, self.n_q + 2 * self.n_kv, self.hd, generator=g, device="cuda") for _ in self.caches]

    def step(self, new, keep, room, qkvs, plan=None, ws=None):
        """One step on the device: a list of outputs, one per layer."""
        c, kvd = self.caches[0], self.kvd
        plan = kvd.paged_plan(c, new, room, keep_len=keep, plan=plan)
        outs, qs = [], []
        for c, x in zip(self.caches, qkvs):
            q = kvd.paged_append(c, plan, x[:, self.n_q:self.n_q + self.n_kv], x[:, self.n_q + self.n_kv:], q=x[:, :self.n_q], rope=self.table)
            outs.append(kvd.paged_attention(q, c, plan, window=self.window, workspace=ws))
            qs.append(q)
        return plan, qs, outs

    def check(self, new, keep, qkvs, plan, qs, outs):
        """The same step by the definition, on what the requests held."""
        torch = self.torch
        at = 0
        for b, n in enumerate(new):
            for layer, x in enumerate(qkvs):
                kept = self.held[layer][b][: keep[b]]
                rows = x[at:at + n].double().cpu().numpy()
                pos = list(range(keep[b], keep[b] + n))
                if n:
                    f = _freqs_yarn(self.hd, 8.0, 256.0)
                    turned = _turn_with(rows[:, : self.n_q + self.n_kv], pos, self.hd, *f)
                    # the rotation itself is checked elsewhere; rounding ties may fall either way, so
                    # attention is checked on the rows that the cache and q hold
                    slots = plan.slots[at:at + n].long()
                    c = self.caches[layer]
                    k = c.k.transpose(1, 2).reshape(-1, self.n_kv, self.hd)[slots]
                    v = c.v.transpose(1, 2).reshape(-1, self.n_kv, self.hd)[slots]
                    step = float(torch.finfo(self.dt).eps)
                    for got, want in ((qs[layer][at:at + n], turned[:, : self.n_q]), (k, turned[:, self.n_q:])):
                        assert float((got.double().cpu() - torch.from_numpy(want)).abs().max()) <= step * (1 + float(np.abs(want).max()))
                    assert torch.equal(v, x[at:at + n, self.n_q + self.n_kv:].to(self.dt))
                    kept = torch.cat([kept, torch.cat([k, v], 1)])
                    want = _attend(torch, qs[layer][at:at + n], kept[:, : self.n_kv], kept[:, self.n_kv:], kept.shape[0], self.hd ** -0.5, self.window)
                    _check_attend(torch, outs[layer][at:at + n], *want, self.dt, 6.0)
                self.held[layer][b] = kept
            at += n


def _freqs_yarn(rot, factor, length):
    i = np.arange(0, rot, 2, dtype=np.float64)
    f = 10000.0 ** (-i / rot)
    dim = lambda turns: rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    low, high = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rot - 1)
    r = np.clip((i / 2 - low) / max(high - low, 1e-3), 0, 1)
    return f / factor * r + f * (1 - r), 0.1 * math.log(factor) + 1


def _turn_with(x, pos, rot, f, mul):
    a = np.array(pos, np.float64)[:, None] * f[None]
    c, s = (np.cos(a) * mul)[:, None], (np.sin(a) * mul)[:, None]
    n = rot // 2
    return np.concatenate([x[..., :n] * c - x[..., n:] * s, x[..., n:] * c + x[..., :n] * s], -1)


STEPS = [([40, 7, 0, 200], None), ([1, 1, 1, 1], None), ([1, 4, 130, 1], None), ([1, 1, 1, 0], [41, 0, 131, 60]), ([3, 300, 1, 90], [0, 1, 132, 60]),
         ([0, 1, 1, 1], None), ([1, 1, 0, 5], [3, 301, 0, 145])]


@pytest.mark.parametrize("dtype,hd,group,page,window", [("bf16", 128, 4, 16, 0), ("f16", 64, 2, 64, 50)])
def test_a_server_runs_steps(env, dtype, hd, group, page, window):
    """Prompts, decode steps, drafts rejected, requests dropped and started again in one batch, over two layers."""
    torch, kvd = env
    s = Server(torch, kvd, 4, 2, group, hd, page, 800 // page + 8, 400 // page + 2, _dt(torch, dtype), window=window)
    now = [0] * 4
    for i, (new, keep) in enumerate(STEPS):
        room = sum(new) + (i % 3) * 5
        x = s.inputs(max(room, 1), 100 + i)
        plan, qs, outs = s.step(_i32(torch, new), None if keep is None else _i32(torch, keep), max(room, 1), x)
        assert s.caches[0].device_error() == 0, i
        s.check(new, list(now) if keep is None else keep, x, plan, qs, outs)
        now = [(a if keep is None else b) + n for a, b, n in zip(now, keep or now, new)]
        assert s.caches[0].seq_len.tolist() == now


def test_a_captured_step_replays_while_lengths_go_on(env):
    """One graph of plan, append and attention, replayed with new numbers in its inputs, against the same steps run eagerly."""
    torch, kvd = env
    room = 420
    make = lambda: Server(torch, kvd, 4, 2, 4, 128, 16, 60, 27, torch.bfloat16, layers=1)  # noqa: E731
    eager, graph = make(), make()
    new, keep = _i32(torch, [0] * 4), _i32(torch, [0] * 4)
    x = graph.inputs(room, 1)
    for i in range(2):  # before the capture: a plan's buffers, and kernels that have run once
        plan, _, _ = graph.step(new, keep, room, x)
    ws = torch.empty(kvd.paged_attention_workspace(room, 8, 2, 128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan, qs, outs = graph.step(new, keep, room, x, plan=plan, ws=ws)
    now = [0] * 4
    for i, (n, k) in enumerate(STEPS):
        k = list(now) if k is None else k
        y = eager.inputs(room, 200 + i)
        new.copy_(_i32(torch, n))
        keep.copy_(_i32(torch, k))
        x[0].copy_(y[0])
        outs[0].fill_(2.0)
        g.replay()
        _, _, want = eager.step(_i32(torch, n), _i32(torch, k), room, y)
        t = sum(n)
        assert torch.equal(outs[0][:t], want[0][:t]) and bool((outs[0][t:] == 2).all()), i
        assert torch.equal(graph.caches[0].seq_len, eager.caches[0].seq_len) and torch.equal(plan.slots[:t], plan.slots[:t])
        now = [a + b for a, b in zip(k, n)]
        assert graph.caches[0].seq_len.tolist() == now and graph.caches[0].device_error() == 0


def test_capture_without_a_workspace(env):
    """A workspace taken by the call itself lives as long as the graph that captured it; small calls (joined in the kernel) and larger
    ones, replayed between eager calls."""
    torch, kvd = env
    for lens, new in (([9000], [1]), ([700, 3000], [40, 90])):
        cache, _ = _poisoned(torch, kvd, lens, 2, 128, 16, torch.bfloat16, 3)
        q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
        plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
        want = kvd.paged_attention(q, cache, plan)
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = kvd.paged_attention(q, cache, plan)
            graphs.append((g, out))
        for _ in range(4):
            for g, out in graphs:
                out.zero_()
                g.replay()
                assert torch.equal(kvd.paged_attention(q, cache, plan), want)
                assert torch.equal(out, want)
        assert cache.device_error() == 0


def test_a_workspace_of_any_contents(env):
    """No initialisation: zeros, ones and what an earlier call of other sizes left give the same bits."""
    torch, kvd = env
    ws = torch.empty(kvd.paged_attention_workspace(300, 8, 2, 128), dtype=torch.uint8, device="cuda")
    first = {}
    for fill in (0, 255, 1, None, None):
        for lens, new in (([9000], [1]), ([700, 3000], [40, 90]), ([20, 30000, 5], [1, 2, 1]), ([2500], [300])):
            cache, _ = _poisoned(torch, kvd, lens, 2, 128, 16, torch.bfloat16, 3)
            q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
            plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
            if fill is not None:
                ws.fill_(fill)
            out = kvd.paged_attention(q, cache, plan, workspace=ws)
            assert cache.device_error() == 0
            assert torch.equal(out, first.setdefault(str(lens), out))


@pytest.mark.parametrize("softcap,scale", [(0.0, 0.09), (30.0, 0.09), (30.0, 9.0)])
@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f16", 64)])
def test_what_nobody_holds_leaves_no_trace(env, dtype, hd, softcap, scale):
    """Rows of pages behind a request's last one and rows of q behind the last request: the same bits whatever they are (they share
    tiles, and warps, with rows that count)."""
    torch, kvd = env
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    for lens, new in (([2001, 77], [1, 1]), ([530, 1000], [3, 150]), ([40], [40])):
        cache, _ = _poisoned(torch, kvd, lens, 2, hd, 64, dt, 11)
        t = sum(new)
        q = torch.randn(t + 5, 10, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(12)).to(dt)
        plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
        free = torch.isnan(cache.k)
        outs = []
        for junk in (0.0, float("nan"), float("inf"), -float("inf"), 60000.0, -60000.0):
            for x in (cache.k, cache.v):
                x.masked_fill_(free, junk)
            q[t:] = junk
            outs.append(kvd.paged_attention(q, cache, plan, scale=scale, softcap=softcap)[:t])
        assert cache.device_error() == 0
        assert not bool(torch.isnan(outs[0]).any())
        assert all(torch.equal(outs[0], x) for x in outs)


def test_two_streams_and_repeats_give_the_same_bits(env):
    torch, kvd = env
    cases = []
    for seed, dt, hd in ((1, torch.bfloat16, 128), (2, torch.float16, 64)):
        cache, _ = _poisoned(torch, kvd, [5000, 300, 77], 2, hd, 16, dt, seed)
        q = torch.randn(203, 8, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dt)
        cases.append((cache, q, kvd.PagedPlan(_i32(torch, [0, 2, 202, 203]), cache.seq_len)))
    alone = [kvd.paged_attention(q, c, p) for c, q, p in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(5):
        for (c, q, p), s, o in zip(cases, streams, outs):
            o.append(kvd.paged_attention(q, c, p, stream=s))
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(a, x) for x in o)


def test_a_failed_launch_is_reported(env):
    torch, kvd = env
    from kv_cache_decode_attention_gb300 import _abi

    cache, _ = _poisoned(torch, kvd, [50], 1, 64, 16, torch.bfloat16, 1)
    cache = kvd.PagedKvCache.of(cache.k, cache.v, cache.block_table, cache.seq_len, _i32(torch, list(range(cache.n_pages))), _i32(torch, [0]))
    x = torch.ones(1, 1, 64, device="cuda", dtype=torch.bfloat16)
    plan = kvd.PagedPlan(_i32(torch, [0, 1]), cache.seq_len, positions=_i32(torch, [0]), slots=_i32(torch, [-1]))
    calls = [(lambda: kvd.rope(x, None, plan.positions, kvd.RopeTable(64)), 1), (lambda: kvd.paged_plan(cache, _i32(torch, [0]), 0), 1),
             (lambda: kvd.paged_append(cache, plan, x, x), 1), (lambda: kvd.paged_attention(x, cache, plan), 1),
             (lambda: kvd.paged_attention(x.expand(20, 1, 64), cache, plan), 2)]
    try:
        for call, launches in calls:
            for n in range(launches):
                assert _abi.lib().kvd_test_fail_after(n) == 0
                with pytest.raises(kvd.KvdError) as e:
                    call()
                assert e.value.status == _abi.ECUDA
            _abi.lib().kvd_test_fail_after(-1)
            call()
    finally:
        _abi.lib().kvd_test_fail_after(-1)
    torch.cuda.synchronize()
    assert cache.device_error() == 0


def test_python_checks(env):
    """What the binding refuses before any call of the library."""
    torch, kvd = env
    cache = kvd.PagedKvCache(4, 16, 2, 64, 2, 2)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    kv = torch.zeros(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    plan = kvd.paged_plan(cache, _i32(torch, [1, 1]), 2)
    bad = [lambda: kvd.paged_plan(cache, _i32(torch, [1]), 2), lambda: kvd.paged_plan(cache, torch.ones(2, device="cuda"), 2),
           lambda: kvd.paged_plan(cache, torch.ones(2, dtype=torch.int32), 2), lambda: kvd.paged_plan(cache, _i32(torch, [1, 1]), -1),
           lambda: kvd.paged_plan(cache, _i32(torch, [1, 1]), 3, plan=plan), lambda: kvd.paged_plan(cache, _i32(torch, [1, 1]), 2, advance=False, plan=plan),
           lambda: kvd.paged_append(cache, plan, kv, kv.float()), lambda: kvd.paged_append(cache, plan, kv[:1], kv[:1]),
           lambda: kvd.paged_append(cache, plan, kv, kv, q=q, q_out=q.float()), lambda: kvd.paged_append(cache, plan, kv.half(), kv.half()),
           lambda: kvd.paged_append(cache, plan, q, q), lambda: kvd.paged_attention(q.half(), cache, plan), lambda: kvd.paged_attention(q[..., :32], cache, plan),
           lambda: kvd.paged_attention(q, cache, plan, sinks=torch.zeros(3, device="cuda")), lambda: kvd.paged_attention(q, cache, plan, scale=0.0),
           lambda: kvd.paged_attention(q, cache, plan, window=-1), lambda: kvd.paged_attention(q, cache, plan, workspace=torch.empty(8, device="cuda")),
           lambda: kvd.paged_attention(q, cache, plan, out=q), lambda: kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, [0, 1]), cache.seq_len)),
           lambda: kvd.RopeTable(64, "halves"), lambda: kvd.RopeTable(64, scaling="none at all"), lambda: kvd.RopeTable(63),
           lambda: kvd.rope(None, None, plan.positions, kvd.RopeTable(64)), lambda: kvd.rope(q, kv.float(), plan.positions, kvd.RopeTable(64)),
           lambda: kvd.rope(q.double(), None, plan.positions, kvd.RopeTable(64)), lambda: kvd.rope(q, None, plan.positions[:1], kvd.RopeTable(64)),
           lambda: kvd.PagedKvCache(4, 24, 2, 64, 2, 2) and kvd.paged_plan(kvd.PagedKvCache(4, 24, 2, 64, 2, 2), _i32(torch, [1, 1]), 2),
           lambda: kvd.PagedKvCache.of(cache.k, cache.v.float(), cache.block_table, cache.seq_len),
           lambda: kvd.PagedKvCache.of(cache.k, cache.v, cache.block_table, cache.seq_len[:1]),
           lambda: kvd.PagedKvCache.of(None, None, cache.block_table, cache.seq_len), lambda: kvd.paged_plan(kvd.PagedKvCache.of(cache.k, cache.v, cache.block_table, cache.seq_len), _i32(torch, [1, 1]), 2)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, kvd.KvdError)):
            f()
            pytest.fail("call %d was taken" % i)
    assert cache.device_error() == 0


def test_lengths_past_31_bits_of_offsets(env):
    """A pool whose byte and element offsets pass 2^32: the rows of its last pages."""
    torch, kvd = env
    if torch.cuda.get_device_properties(0).total_memory < 60e9:
        pytest.skip("needs 40 GB")
    n_pages, page, n_kv, hd = 40000, 128, 4, 128  # 2.6e9 elements each of K and V
    k = torch.empty(n_pages, n_kv, page, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    table = _i32(torch, [[n_pages - 1, 5, n_pages - 3, 0], [n_pages - 2, 0, 0, 0]])
    cache = kvd.PagedKvCache.of(k, v, table, _i32(torch, [300, 2]))
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(302, 2 * n_kv, hd, generator=g, device="cuda").bfloat16()
    pos = list(range(300)) + [0, 1]
    slot = [int(table[0, p // 128]) * 128 + p % 128 for p in range(300)] + [(n_pages - 2) * 128, (n_pages - 2) * 128 + 1]
    plan = kvd.PagedPlan(_i32(torch, [0, 300, 302]), cache.seq_len, positions=_i32(torch, pos), slots=_i32(torch, slot))
    kvd.paged_append(cache, plan, rows[:, :n_kv], rows[:, n_kv:])
    q = torch.randn(302, n_kv, hd, generator=g, device="cuda").bfloat16()
    out = kvd.paged_attention(q, cache, plan)
    assert cache.device_error() == 0
    for a, e in ((0, 300), (300, 302)):
        _check_attend(torch, out[a:e], *_attend(torch, q[a:e], rows[a:e, :n_kv], rows[a:e, n_kv:], e - a, hd ** -0.5), torch.bfloat16, 6.0)


# Caps far above the scores, where tanh(y) is y to the last bit; around them, where the coefficients of its polynomial in powers of the score
# leave the f32 range one by one; and below the scores, where it saturates.
CAPS = [(1e3, None), (1e4, None), (2e4, None), (5e4, None), (1e6, None), (1e10, None), (1e15, None), (1e30, None), (2e38, None), (30.0, 1e-4), (120.0, 1e-3),
        (1.2e3, 1 / 128), (30.0, 9.0), (100.0, 9.0), (5.0, 2.0), (1e-3, 0.1), (1e-22, 1e-23), (1e20, 1e-19)]


@pytest.mark.parametrize("softcap,scale", CAPS)
@pytest.mark.parametrize("hd,dtype", [(64, "f16"), (128, "bf16")])
def test_attention_with_a_cap_of_any_size(env, hd, dtype, softcap, scale):
    """Single tokens, prompts and chunks, with and without a window.  tanh moves a score's error by no more than itself and adds, with
    the products and sums in log2 units behind it, 2^-19 of the capped score (2^-21 of the special functions' form from |y| = 1/2 on,
    2^-22 of the polynomial below, 2^-23 each of the argument, the product with the cap and the difference to the maximum)."""
    torch, kvd = env
    dt = _dt(torch, dtype)
    scale = hd ** -0.5 if scale is None else scale
    for window in (0, 100):
        for lens, new in (([900, 1, 130, 2000, 64], [1, 1, 130, 300, 3]), ([77], [1])):
            cache, rows = _poisoned(torch, kvd, lens, 2, hd, 16, dt, 81)
            q = (torch.randn(sum(new), 8, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(82)) * 1.5).to(dt)
            plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
            out = kvd.paged_attention(q, cache, plan, scale=scale, window=window, softcap=softcap)
            assert cache.device_error() == 0
            at = 0
            for (kk, vv), total, n in zip(rows, lens, new):
                x = q[at:at + n]
                # the definition without the cap's own slack, and that of the capped scores in its place
                want, size, _ = _attend(torch, x, kk, vv, total, scale, window, softcap)
                raw = torch.einsum("nhd,thd->hnt", x.double(), kk.repeat_interleave(4, 1).double()) * scale
                moved = hd * 2.0 ** -24 * scale * torch.einsum("nhd,thd->hnt", x.double().abs(), kk.repeat_interleave(4, 1).double().abs())
                slack = 2 * (moved + 2.0 ** -19 * (softcap * torch.tanh(raw / softcap)).abs()).amax(-1).T[..., None] + 2.0 ** -20
                _check_attend(torch, out[at:at + n], want, size, slack, dt, float(vv.abs().max()))
                at += n


def test_attention_with_a_cap_below_the_scale_and_scores_of_zero(env):
    """Coefficients past the f32 range: a score of zero stays one."""
    torch, kvd = env
    cache, rows = _poisoned(torch, kvd, [300, 40], 2, 64, 16, torch.bfloat16, 83)
    plan = kvd.PagedPlan(_i32(torch, [0, 30, 31]), cache.seq_len)
    q = torch.zeros(31, 4, 64, device="cuda", dtype=torch.bfloat16)
    out = kvd.paged_attention(q, cache, plan, scale=1e10, softcap=1.0)
    assert cache.device_error() == 0
    for (a, e), (kk, vv) in zip(((0, 30), (30, 31)), rows):
        _check_attend(torch, out[a:e], *_attend(torch, q[a:e], kk, vv, kk.shape[0], 1.0), torch.bfloat16, float(vv.abs().max()))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
def test_a_window_wider_than_any_cache_is_none(env, window):
    """Also where the first new rows stand before the start of their request."""
    torch, kvd = env
    lens, new = [3, 0, 130, 0, 700], [5, 2, 400, 1, 1]
    assert torch.equal(*(_run_attend(torch, kvd, lens, new, 2, 4, 128, 16, torch.bfloat16, 91, window=w)[: sum(new)] for w in (window, 0)))


@pytest.mark.parametrize("lens,new", [([9000], [1]), ([60000, 300], [1, 1]), ([20, 30000, 5], [1, 2, 1]), ([2500, 900], [300, 100])])
def test_a_launch_given_up_leaves_no_trace(env, lens, new):
    """One CTA's waits end early, at one moment or another: the error bit, every ticket of the workspace back at zero, and the next calls and
    replays right.  A graph's replays all come with the same tickets."""
    torch, kvd = env
    from kv_cache_decode_attention_gb300 import _abi

    cache, _ = _poisoned(torch, kvd, lens, 2, 128, 16, torch.bfloat16, 3)
    q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
    ws = torch.zeros(kvd.paged_attention_workspace(sum(new), 8, 2, 128), dtype=torch.uint8, device="cuda")
    counts = ws[: 152 * 8].view(torch.int64)
    want, out = kvd.paged_attention(q, cache, plan, workspace=ws), torch.empty_like(q)
    assert cache.device_error() == 0
    gave_up = 0
    try:
        for cta in (0, 37, 75, 76, 151):
            for after in (0, 2000, 5000, 9000):
                assert _abi.lib().kvd_test_give_up(cta, after) == 0
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    kvd.paged_attention(q, cache, plan, out=out, workspace=ws)
                _abi.lib().kvd_test_give_up(-1, 0)
                for _ in range(4):
                    out.fill_(float("nan"))
                    graph.replay()
                    error = cache.device_error()
                    assert error in (0, 1)
                    gave_up += error
                    assert not bool((counts & 255).any()), (cta, after)
                    assert error == 1 or torch.equal(out, want)
                assert torch.equal(kvd.paged_attention(q, cache, plan, out=out, workspace=ws), want) and cache.device_error() == 0
    finally:
        _abi.lib().kvd_test_give_up(-1, 0)
    assert gave_up >= 4


def test_outputs_made_for_another_stream_are_its_own(env):
    """With stream= and no outputs given, a call's new outputs are not taken from memory that the current stream has just let go of and is
    still reading; and what the current stream does with them holds them, though it has dropped them."""
    torch, kvd = env
    side, tokens = torch.cuda.Stream(), 1 << 15
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = kvd.PagedKvCache(tokens // 16, 16, 1, 64, 1, tokens // 16)
    x = torch.randn(tokens, 2, 64, device="cuda", generator=g).bfloat16()
    q, k, new = x, x[:, :1], _i32(torch, [tokens])
    table, pos = kvd.RopeTable(64), torch.arange(tokens, device="cuda", dtype=torch.int32)
    plan = kvd.paged_plan(cache, new, tokens)
    kvd.paged_append(cache, plan, k, k)
    empty = kvd.PagedPlan(plan.cu_new.zero_(), plan.seq_len)  # an attention of no rows writes nothing
    other = kvd.PagedKvCache(tokens // 16, 16, 1, 64, 1, tokens // 16)
    calls = [("rope", lambda: list(kvd.rope(q, k, pos, table, stream=side))),
             ("plan", lambda: [getattr(kvd.paged_plan(other, new, tokens, advance=False, stream=side), n) for n in ("positions", "slots")]),
             ("append", lambda: [kvd.paged_append(cache, plan, k, k, q=q, stream=side)]),
             ("attention", lambda: [kvd.paged_attention(q, cache, empty, stream=side)])]
    torch.cuda.synchronize()
    for name, call in calls:
        for _ in range(2):
            outs = call()
            torch.cuda.synchronize()
            like = [torch.empty_like(o, memory_format=torch.contiguous_format).fill_(7) for o in outs]
            shapes = [(o.shape, o.dtype) for o in like]
            del outs
            torch.cuda.synchronize()
            torch.cuda._sleep(20_000_000)
            copies = [t.clone() for t in like]
            held = {t.data_ptr() for t in like}
            del like
            outs = call()
            assert not held & {o.data_ptr() for o in outs}, name
            again = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes]
            assert held & {o.data_ptr() for o in again}, name  # the test would see it
            torch.cuda.synchronize()
            assert all(bool((c == 7).all()) for c in copies), name
            # the caller's work on them, queued behind a wait, outlives its hold on them
            torch.cuda._sleep(20_000_000)
            seen = [o.clone() for o in outs]
            want = [o.data_ptr() for o in outs]
            del outs
            with torch.cuda.stream(side):
                late = [torch.empty(s, dtype=d, device="cuda") for s, d in shapes]
            assert not set(want) & {o.data_ptr() for o in late}, name
            torch.cuda.synchronize()
            del again, late, copies, seen
    assert cache.device_error() == 0 and other.device_error() == 0


def test_attention_refuses_outputs_that_share_memory(env):
    """A slice of q's own array shifted by a head or a token, q itself, rows on one another, the pages; slices beside q are taken."""
    torch, kvd = env
    cache, _ = _poisoned(torch, kvd, [300, 40], 2, 64, 16, torch.bfloat16, 61)
    x = torch.randn(31, 17, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    old = x.clone()
    q, plan = x[:30, :8, :64], kvd.PagedPlan(_i32(torch, [0, 20, 30]), cache.seq_len)
    flat = torch.empty(30 * 8 * 64, device="cuda", dtype=torch.bfloat16)
    for bad in (q, x[:30, 1:9, :64], x[1:, :8, :64], x[:30, 7:15, 32:96], torch.as_strided(flat, (30, 8, 64), (64, 64, 1)),
                torch.as_strided(flat, (30, 8, 64), (256, 32, 1)), cache.k.view(-1)[: 30 * 512].view(30, 8, 64), cache.v.view(-1)[-30 * 512:].view(30, 8, 64)):
        with pytest.raises(kvd.KvdError):
            kvd.paged_attention(q, cache, plan, out=bad)
    assert torch.equal(x, old)
    want = kvd.paged_attention(q.contiguous(), cache, plan)
    flipped = torch.empty(8, 30, 64, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    for out in (x[:30, 8:16, :64], x[:30, :8, 64:], x[:30, 9:, 64:], flipped):
        assert torch.equal(kvd.paged_attention(q, cache, plan, out=out), want)
        assert torch.equal(q, old[:30, :8, :64])
    assert cache.device_error() == 0


def test_rotated_outputs_beside_their_inputs(env):
    """Slices of one projection that are taken as outputs, and those that are refused, with the arrays as they were."""
    torch, kvd = env
    x = torch.randn(40, 24, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9)).bfloat16()
    old, pos, table = x.clone(), torch.arange(40, device="cuda", dtype=torch.int32), kvd.RopeTable(64)
    q, k = x[:, :8], x[:, 8:12]
    want = kvd.rope(q, k, pos, table)
    got = kvd.rope(q, k, pos, table, q_out=x[:, 12:20], k_out=x[:, 20:])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(x[:, :12], old[:, :12])
    half = kvd.rope(q[..., :64], None, pos, table, q_out=q[..., 64:])[0]
    assert torch.equal(half, want[0][..., :64])
    x.copy_(old)
    flat = torch.empty(40 * 8 * 128, device="cuda", dtype=torch.bfloat16)
    for bad in (dict(q_out=x[:, 1:9]), dict(q_out=x[:, 8:16]), dict(k_out=x[:, 7:11]), dict(q_out=q, k_out=x[:, 4:8]),
                dict(q_out=torch.as_strided(flat, (40, 8, 128), (64, 128, 1))), dict(q_out=x[:, 12:20], k_out=x[:, 16:20])):
        with pytest.raises(kvd.KvdError):
            kvd.rope(q, k, pos, table, **bad)
    cache = kvd.PagedKvCache(8, 16, 4, 128, 1, 8)
    plan = kvd.paged_plan(cache, _i32(torch, [40]), 40)
    same = kvd.PagedKvCache.of(cache.k, cache.k, cache.block_table, cache.seq_len)
    rows = cache.k.view(-1)[: 40 * 512].view(40, 4, 128)
    for call in (lambda: kvd.paged_append(cache, plan, k, k, q=q, q_out=x[:, 4:12]), lambda: kvd.paged_append(same, plan, k, k),
                 lambda: kvd.paged_append(cache, plan, k, rows), lambda: kvd.paged_append(cache, plan, rows, k)):
        with pytest.raises(kvd.KvdError):
            call()
    assert torch.equal(x, old)
    kvd.paged_append(cache, plan, k, k, q=q, q_out=x[:, 12:20])
    assert torch.equal(x[:, 12:20], old[:, :8]) and cache.device_error() == 0


@pytest.mark.parametrize("n_seq,rows", [(3, 40), (700, 60), (3000, 20)])
@pytest.mark.parametrize("bad", [-1, "n_pages", 2 ** 31 - 1])
def test_plan_refuses_pages_outside_the_pool(env, n_seq, rows, bad):
    """Among those given back and among those taken: the step changes nothing, and goes through once the number is put right."""
    torch, kvd = env
    r = np.random.default_rng(n_seq)
    width = -(-2 * rows // 16)
    n_pages = n_seq * width
    bad = n_pages if bad == "n_pages" else bad
    cache = kvd.PagedKvCache(n_pages, 16, 1, 64, n_seq, width)
    model = Model(n_seq, 16, width, n_pages)
    first = r.integers(1, rows, n_seq).tolist()
    assert model.step(first, None, sum(first)) is not None
    kvd.paged_plan(cache, _i32(torch, first), sum(first))
    _same_state(cache, model)
    keep = [0 if b % 3 == 0 else n for b, n in enumerate(model.len)]
    new = r.integers(0, rows, n_seq).tolist()
    after = [-(-(k + n) // 16) for k, n in zip(keep, new)]
    gives = [b for b in range(n_seq) if after[b] < len(model.pages[b])]
    if not gives:  # a small batch: the first gives back what it has
        new[0], gives = 0, [0]
        after[0] = 0
    room, takes, given = sum(new), sum(max(0, a - len(p)) for a, p in zip(after, model.pages)), sum(max(0, len(p) - a) for a, p in zip(after, model.pages))
    places = [(cache.block_table, (b, int(r.integers(after[b], len(model.pages[b]))), )) for b in (gives[0], gives[-1])]
    if takes > given:  # below the height that stands, as far as the step digs
        places += [(cache.free_pages, (int(cache.n_free) - 1,)), (cache.free_pages, (int(cache.n_free) - (takes - given),))]
    for tensor, at in places:
        good = int(tensor[at])
        tensor[at] = bad
        state = [t.clone() for t in (cache.seq_len, cache.n_free, cache.block_table)]
        height = int(cache.n_free)
        stack = cache.free_pages[:height].clone()
        for advance in (False, True):
            plan = kvd.paged_plan(cache, _i32(torch, new), room, keep_len=_i32(torch, keep), advance=advance)
            assert cache.device_error() == 2
            assert not plan.cu_new.any() and bool((plan.slots == -1).all()) and bool((plan.positions == -1).all())
            assert torch.equal(plan.seq_len, state[0]) and torch.equal(plan.n_free, state[1])
            for a, b in zip(state, (cache.seq_len, cache.n_free, cache.block_table)):
                assert torch.equal(a, b)
            assert torch.equal(cache.free_pages[:height], stack)
        tensor[at] = good
    # a wrong page below those taken, or kept with room to spare, is no part of the step
    if takes < given + int(cache.n_free):
        cache.free_pages[0], spare = bad, int(cache.free_pages[0])
    want = model.step(new, keep, room)
    plan = kvd.paged_plan(cache, _i32(torch, new), room, keep_len=_i32(torch, keep))
    assert cache.device_error() == 0 and plan.slots.tolist() == want[2] and plan.positions.tolist() == want[1]
    if len(model.free) and model.free[0] != int(cache.free_pages[0]):
        cache.free_pages[0] = spare
    _same_state(cache, model)


def test_the_error_word_waits_for_every_stream(env):
    """A call still under way on another stream is in the word, and the word is clear for the next one."""
    torch, kvd = env
    cache = kvd.PagedKvCache(2, 16, 2, 64, 1, 2)
    x = torch.ones(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    bad = kvd.PagedPlan(None, None, positions=_i32(torch, [0]), slots=_i32(torch, [32]))
    good = kvd.PagedPlan(None, None, positions=_i32(torch, [0]), slots=_i32(torch, [31]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for plan, word in ((bad, 2), (good, 0), (bad, 2), (bad, 2), (good, 0)):
        with torch.cuda.stream(side):
            torch.cuda._sleep(30_000_000)
            kvd.paged_append(cache, plan, x, x)
        assert cache.device_error(clear=False) == word and cache.device_error() == word and cache.device_error() == 0


def test_few_busy_places_among_many(env):
    """The most places a call takes, all but three of them without new rows: at both ends and in the middle."""
    torch, kvd = env
    n = 1 << 20
    lens, busy = [300, 40, 700], [0, n // 2 + 7, n - 1]
    small, rows = _poisoned(torch, kvd, lens, 2, 64, 16, torch.bfloat16, 61)
    table = torch.full((n, small.max_pages), -1, dtype=torch.int32, device="cuda")
    table[busy] = small.block_table
    seq, new = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
    seq[busy], new[busy] = small.seq_len, _i32(torch, [1, 30, 2])
    cu = torch.cat([new[:1] * 0, new.cumsum(0, dtype=torch.int32)])
    cache = kvd.PagedKvCache.of(small.k, small.v, table, seq)
    q = torch.randn(33, 8, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).bfloat16()
    out = kvd.paged_attention(q, cache, kvd.PagedPlan(cu, seq))
    assert torch.equal(out, kvd.paged_attention(q, small, kvd.PagedPlan(_i32(torch, [0, 1, 31, 33]), small.seq_len)))
    assert cache.device_error() == 0 and small.device_error() == 0


def test_a_plan_apart_may_not_hold_a_view_of_the_state(env):
    torch, kvd = env
    cache = kvd.PagedKvCache(8, 16, 1, 64, 2, 4)
    new = _i32(torch, [20, 3])
    apart = kvd.paged_plan(cache, new, 23, advance=False)
    for plan in (kvd.PagedPlan(apart.cu_new, cache.seq_len[:], apart.n_free, apart.positions, apart.slots),
                 kvd.PagedPlan(apart.cu_new, apart.seq_len, cache.n_free.view(1, 1), apart.positions, apart.slots)):
        with pytest.raises(ValueError):
            kvd.paged_plan(cache, new, 23, advance=False, plan=plan)
    assert cache.seq_len.tolist() == [0, 0] and int(cache.n_free) == 8
    again = kvd.paged_plan(cache, new, 23, advance=False, plan=apart)
    assert again is apart and apart.seq_len.tolist() == [20, 3] and cache.seq_len.tolist() == [0, 0] and cache.device_error() == 0


def test_a_replayed_plan_equals_an_eager_one(env):
    """What the captured step's plan holds after each replay: slots, positions, row counts, tables, the stack, and -1 behind the last row."""
    torch, kvd = env
    room = 420
    eager, graph = (kvd.PagedKvCache(60, 16, 2, 64, 4, 27) for _ in range(2))
    new, keep = _i32(torch, [0] * 4), _i32(torch, [0] * 4)
    plan = kvd.paged_plan(graph, new, room, keep_len=keep)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvd.paged_plan(graph, new, room, keep_len=keep, plan=plan)
    now, model = [0] * 4, Model(4, 16, 27, 60)
    for n, k in STEPS + [([0, 0, 0, 0], [0, 0, 0, 0]), ([400, 0, 3, 17], None)]:
        k = list(now) if k is None else k
        new.copy_(_i32(torch, n))
        keep.copy_(_i32(torch, k))
        for t in (plan.slots, plan.positions, plan.cu_new):
            t.fill_(77)
        g.replay()
        other = kvd.paged_plan(eager, _i32(torch, n), room, keep_len=_i32(torch, k))
        cu, pos, slots = model.step(n, k, room)
        for p in (plan, other):
            assert p.cu_new.tolist() == cu and p.positions.tolist() == pos + [-1] * (room - cu[-1]) and p.slots.tolist() == slots + [-1] * (room - cu[-1])
        for c in (graph, eager):
            _same_state(c, model)
            assert c.device_error() == 0
        now = [a + b for a, b in zip(k, n)]


def test_a_step_captured_onto_another_stream(env):
    """Plan, append and attention captured with stream=, new outputs each, and two such graphs on one workspace, replayed in turn: small
    calls, which join their pieces by tickets in it, and larger ones."""
    torch, kvd = env
    made = []
    for lens, new, seed in (([9000, 5], [1, 1], 3), ([700, 3000], [40, 90], 4)):
        cache, _ = _poisoned(torch, kvd, lens, 2, 128, 16, torch.bfloat16, seed)
        plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
        q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()
        made.append((cache, plan, q))
    small = kvd.PagedKvCache(40, 16, 2, 128, 2, 40)
    new, pos = _i32(torch, [300, 20]), torch.arange(130, device="cuda", dtype=torch.int32)
    rows = torch.randn(320, 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    table, ws = kvd.RopeTable(128), torch.empty(kvd.paged_attention_workspace(320, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def step(stream, shared):
        outs = [kvd.paged_attention(q, c, p, workspace=ws if shared else None, stream=stream) for c, p, q in made]
        outs += [kvd.rope(q[:130], None, pos[: q.shape[0]], table, stream=stream)[0] for _, _, q in made]
        p = kvd.paged_plan(small, new, 330, keep_len=_zero, stream=stream)
        qr = kvd.paged_append(small, p, rows_k, rows_k, q=rows_q, rope=table, stream=stream)
        return outs + [p.slots, p.positions, p.cu_new, kvd.paged_attention(qr, small, p, workspace=ws_big if shared else None, stream=stream)[:320]]

    _zero = _i32(torch, [0, 0])
    rows = torch.cat([rows, rows[:10]])
    rows_q, rows_k = rows, rows[:, :2]
    ws_big = torch.empty(kvd.paged_attention_workspace(330, 8, 2, 128), dtype=torch.uint8, device="cuda")
    want = step(None, False)
    torch.cuda.synchronize()
    graphs = []
    for shared in (True, True, False):
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            outs = step(side, shared)
            torch.cuda.current_stream().wait_stream(side)
        graphs.append((g, outs))
    for _ in range(3):
        for g, outs in graphs:
            for t in outs:
                t.fill_(9)
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert small.device_error() == 0 and all(c.device_error() == 0 for c, _, _ in made)
