"""Pages of 8-bit codes on the GPU: written, read back and attended, against plain references in 64 bits.

Tolerances, from the arithmetic:
- codes and scales of rows that are not rotated are equal, byte by byte: x / s is exact for a power of two, and a code is x / s
  rounded to nearest even, by the definition below.
- rotated rows carry the rotation's error r (16 * 2^-24 of (|a| + |b|), as for the 16-bit pages), which may move a code by one
  step: off by half a step of e4m3 (2^-4 of the value, at least half of 2^-9 s) of a value that r may have moved: 2^-4 (|x| + r) + 2^-10 s + r.
- reading: code times scale is exact in f32 (28 bits of mantissa and less for scales that are powers of two) or one rounding of it, then one
  rounding to the output's type.
- attention: as for the 16-bit pages (weights rounded to q's type, scores' f32 sums, one rounding of the output), and beside that: q is
  held to 2^-17 of its row's largest, which moves a score by 2^-17 max|q| sum |k| scale; a weight, with its block's scale, is held to
  2^-22 of the largest of its 128 rows, of which the output feels 128 * 2^-22 * 448 max(v_scale) at most.
"""

import math

import numpy as np
import pytest
from test_gpu_paged import _check_attend, _dt, _freqs, _i32, _tiny, _turn

pytestmark = pytest.mark.gpu

LOW, HIGH = 2.0 ** -64, 2.0 ** 64


@pytest.fixture(scope="module")
def env():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import kv_cache_decode_attention_gb300 as kvd
    from kv_cache_decode_attention_gb300.build import build

    build()
    return torch, kvd


# ---------------------------------------------------------------- the definition

# the 127 finite magnitudes of e4m3 by their codes, and the borders between them
MAGNITUDES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def _codes(y):
    """Codes of f64 values: the nearest magnitude, ties to the even code, 448 at most; NaN is 0x7f."""
    a = np.minimum(np.abs(y), 448.0)
    i = np.clip(np.searchsorted(MAGNITUDES, a, side="right") - 1, 0, 125)
    lo, hi = MAGNITUDES[i], MAGNITUDES[i + 1]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    c = np.where(np.isnan(y), 127, i + up).astype(np.uint8)
    return np.where(np.signbit(y) & ~np.isnan(y), c | 128, c).astype(np.uint8)


def _values(codes):
    m = np.append(MAGNITUDES, np.nan)[codes & 127]
    return np.where(codes & 128, -m, m)


def _need(top):
    s = LOW
    while 448.0 * s < top and s < HIGH:
        s *= 2
    return s


class Model:
    """Pages on the host: codes [n_pages, n_kv, page, hd] and scales, by the definition."""

    def __init__(self, codes, scale):
        self.codes, self.scale = codes.copy(), scale.astype(np.float64).copy()

    def write(self, slots, rows):
        size = self.codes.shape[2]
        at = 0
        while at < len(slots):
            if slots[at] < 0 or slots[at] >= size * self.codes.shape[0]:
                at += 1
                continue
            end = at + 1
            while end < len(slots) and slots[end] == slots[end - 1] + 1 and slots[end] % size:
                end += 1
            p, r0, n = slots[at] // size, slots[at] % size, end - at
            for h in range(self.codes.shape[1]):
                x = rows[at:end, h]
                fine = np.abs(x[np.isfinite(x)])
                need, old = _need(fine.max() if fine.size else 0.0), self.scale[p, h]
                if r0 and old >= need:
                    need = old
                elif r0:
                    self.codes[p, h, :r0] = _codes(_values(self.codes[p, h, :r0]) * np.float64(np.float32(old) / np.float32(need)))
                self.scale[p, h] = need
                self.codes[p, h, r0:r0 + n] = _codes(x / need)
            at = end


def _same(torch, cache, k, v, what=""):
    for codes, scale, model in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        assert np.array_equal(scale.double().cpu().numpy(), model.scale), what
        got = codes.view(torch.uint8).cpu().numpy()
        # (a NaN keeps no sign)
        nan = (got & 127) == 127
        assert np.array_equal(nan, (model.codes & 127) == 127), what
        # zeros may carry either sign
        assert np.array_equal(np.where(nan | ((got & 127) == 0), 0, got), np.where(nan | ((model.codes & 127) == 0), 0, model.codes)), what


def _cache(torch, kvd, n_pages, page, n_kv, hd, n_seq=1, width=None, seed=0):
    """A cache whose pages hold random bytes and scales that nobody wrote."""
    cache = kvd.PagedKvCache(n_pages, page, n_kv, hd, n_seq, width or n_pages, dtype=torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(1000 + seed)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (cache.k_scale, cache.v_scale):
        t.copy_(torch.exp2(torch.randint(-9, 3, t.shape, generator=g, device="cuda").float()))
    return cache


def _models(torch, cache):
    return tuple(Model(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))


def _plan(torch, kvd, positions, slots):
    return kvd.PagedPlan(None, None, positions=_i32(torch, positions), slots=_i32(torch, slots))


# ---------------------------------------------------------------- writing


@pytest.mark.parametrize("given", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hd,page,n_kv", [(64, 16, 3), (128, 16, 8), (128, 32, 1), (64, 128, 2), (128, 128, 5), (128, 64, 2)])
def test_codes_and_scales_are_the_definitions(env, given, hd, page, n_kv):
    """Steps of every length into several requests' pages, in pieces, with rows that outgrow the scale of those before them."""
    torch, kvd = env
    n_pages = 24
    cache = _cache(torch, kvd, n_pages, page, n_kv, hd)
    k, v = _models(torch, cache)
    r = np.random.RandomState(hd + page + n_kv)
    order = r.permutation(n_pages)
    first, at = [order[:8], order[8:16], order[16:]], [0, 0, 0]
    for step, news in enumerate([(1, 0, page), (1, 17, 1), (3, page + 5, 2), (1, 1, 1), (2 * page + 3, 1, 0), (1, 40, page - 1), (5, 1, 33), (1, 1, 1)]):
        pos, slots = [], []
        for b, n in enumerate(news):
            n = min(n, 8 * page - at[b])
            p = np.arange(at[b], at[b] + n)
            pos += p.tolist()
            slots += (first[b][p // page] * page + p % page).tolist()
            at[b] += n
        g = torch.Generator(device="cuda").manual_seed(step)
        x = torch.randn(len(slots) + 2, 2 * n_kv, hd, generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-3, 4, x.shape[:2], generator=g, device="cuda").float() + step * (step % 3)).unsqueeze(-1)
        x = x.to(_dt(torch, given))
        assert kvd.paged_append(cache, _plan(torch, kvd, pos + [-1, -1], slots + [-1, -1]), x[:, :n_kv], x[:, n_kv:]) is None
        host = x.double().cpu().numpy()
        k.write(slots, host[:, :n_kv])
        v.write(slots, host[:, n_kv:])
        _same(torch, cache, k, v, step)
    assert cache.device_error() == 0


def test_values_at_the_edges(env):
    """Ties, subnormals, zeros, infinities and NaN, the smallest and the largest scale, rows behind scales that others gave."""
    torch, kvd = env
    hd, page = 64, 16
    x = torch.zeros(12, 1, hd, device="cuda")
    borders = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
    x[0, 0] = torch.tensor(np.append(borders[:63], 448.0)).float()
    x[1, 0] = torch.tensor(-np.append(borders[63:], 448.0)).float()
    x[2, 0, :6] = torch.tensor([math.inf, -math.inf, math.nan, 1.0, -2.0 ** -10, 3e-39])
    x[3, 0, :3] = torch.tensor([1.75 * 2.0 ** 5, 0.1, -1e-30])
    x[4, 0, :3] = torch.tensor([math.nextafter(1.75 * 2.0 ** 5, 100), 0.1, -1e-30]).float()
    x[4, 0, 0] = torch.nextafter(torch.tensor(1.75 * 2.0 ** 5), torch.tensor(100.0))
    x[6, 0, :2] = torch.tensor([3e38, -1.0])
    x[7, 0, :2] = torch.tensor([1e-42, -1e-25])
    x[8, 0] = math.inf
    x[9, 0] = math.nan
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        y = x.to(dt)
        cache = _cache(torch, kvd, 16, page, 1, hd, seed=3)
        k, v = _models(torch, cache)
        slots = [p * page for p in range(12)]  # each row begins a page of its own
        kvd.paged_append(cache, _plan(torch, kvd, [0] * 12, slots), y, y.flip(0))
        k.write(slots, y.double().cpu().numpy())
        v.write(slots, y.flip(0).double().cpu().numpy())
        _same(torch, cache, k, v, dt)
        slots = [p * page + 1 for p in range(12)]  # and now beside one another, in another order
        y = y.roll(5, 0)
        kvd.paged_append(cache, _plan(torch, kvd, [1] * 12, slots), y, y)
        k.write(slots, y.double().cpu().numpy())
        v.write(slots, y.double().cpu().numpy())
        _same(torch, cache, k, v, dt)
        assert cache.device_error() == 0
    # a scale that is no power of two stays while it is large enough, and is left for one that is
    cache = _cache(torch, kvd, 2, page, 1, hd, seed=4)
    cache.k_scale.fill_(0.3)
    cache.v_scale.fill_(0.003)
    k, v = _models(torch, cache)
    y = torch.randn(2, 1, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 9
    kvd.paged_append(cache, _plan(torch, kvd, [3, 9], [3, page + 9]), y, y)
    host = y.double().cpu().numpy()
    k.write([3, page + 9], host)
    v.write([3, page + 9], host)
    # x / 0.3 is rounded to f32 before it is rounded to a code: only borders may tell
    k.codes[[0, 1], 0, [3, 9]] = _codes((y[:, 0].cpu().numpy() / np.float32(0.3)).astype(np.float64))
    # c * (0.003 / s) likewise
    s = np.float32(v.scale[0, 0])
    before = _cache(torch, kvd, 2, page, 1, hd, seed=4).v.view(torch.uint8).cpu().numpy()
    for p, n in ((0, 3), (1, 9)):
        s = np.float32(v.scale[p, 0])
        assert s > 0.003
        v.codes[p, 0, :n] = _codes((_values(before[p, 0, :n]).astype(np.float32) * (np.float32(0.003) / s)).astype(np.float64))
    _same(torch, cache, k, v)
    assert cache.device_error() == 0
    # a scale that cannot be one: told, and the block goes on with the new rows'
    for bad in (0.0, math.nan, math.inf, -1.0, 2.0 ** -65, 2.0 ** 65):
        cache.k_scale.fill_(bad)
        kvd.paged_append(cache, _plan(torch, kvd, [3], [3]), y[:1], y[:1])
        assert cache.device_error() == 2 and float(cache.k_scale[0, 0]) == _need(float(y[0].abs().max()))


def test_bad_slots_and_no_rows(env):
    torch, kvd = env
    cache = _cache(torch, kvd, 3, 16, 2, 64)
    k, v = _models(torch, cache)
    x = torch.randn(9, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    slots = [48, 47, -5, 2 ** 31 - 1, 14, 15, 16, 17, 49]  # a run ends with its page
    kvd.paged_append(cache, _plan(torch, kvd, list(range(9)), slots), x, x)
    k.write(slots, x.double().cpu().numpy())
    v.write(slots, x.double().cpu().numpy())
    _same(torch, cache, k, v)
    assert cache.device_error() == 2 and cache.device_error() == 0
    kvd.paged_append(cache, _plan(torch, kvd, [], []), x[:0], x[:0])
    kvd.paged_append(cache, _plan(torch, kvd, [0] * 9, [-1] * 9), x, x)
    _same(torch, cache, k, v)


@pytest.mark.parametrize("given,to", [("f32", "bf16"), ("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("hd,rot,layout", [(128, 128, "half"), (128, 64, "interleaved"), (64, 64, "interleaved"), (128, 70, "half"), (64, 6, "interleaved"), (64, 32, "half")])
def test_rotated_rows(env, given, to, hd, rot, layout):
    """Slices of one projection, rows whose starts lie anywhere, lengths around a CTA's 16 tokens; q beside k and v."""
    torch, kvd = env
    for tokens, odd in ((1, 0), (15, 0), (33, 0), (150, 0), (37, 1)):
        n_q, n_kv, page = 6, 2, 32
        cache = _cache(torch, kvd, 8, page, n_kv, hd, seed=tokens)
        g = torch.Generator(device="cuda").manual_seed(tokens)
        wide = torch.randn(tokens, n_q + 2 * n_kv, hd + odd, generator=g, device="cuda").to(_dt(torch, given))
        qkv = wide[..., odd:]
        start = 21
        pos = np.arange(start, start + tokens) + 1000
        slots = np.arange(start, start + tokens)
        plan = _plan(torch, kvd, pos, slots)
        q_out = torch.full((tokens, n_q, hd), 7.0, device="cuda", dtype=_dt(torch, to))
        before = _models(torch, cache)
        q = kvd.paged_append(cache, plan, qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:], q=qkv[:, :n_q], q_out=q_out, rope=kvd.RopeTable(rot, layout))
        assert q is q_out and cache.device_error() == 0
        x = qkv.double().cpu().numpy()
        want, size = _turn(x, pos, rot, layout, "none")
        half = float(torch.finfo(q.dtype).eps) / 2
        slip = size * 16 * 2.0 ** -24
        assert np.all(np.abs(q.double().cpu().numpy() - want[:, :n_q]) <= half * np.abs(want[:, :n_q]) + slip[:, :n_q] * (1 + half) + _tiny(torch, q.dtype))
        k, v = kvd.paged_read(kvd.PagedKvCache.of(cache.k, cache.v, _i32(torch, [list(range(8))]), _i32(torch, [start + tokens]), k_scale=cache.k_scale,
                                                  v_scale=cache.v_scale), _i32(torch, [0, tokens]), tokens, start=_i32(torch, [start]), dtype=torch.float32)
        s = cache.k_scale.double().cpu().numpy()[slots // page][:, :, None]
        wk, rk = want[:, n_q:n_q + n_kv], slip[:, n_q:n_q + n_kv]
        assert np.all(np.abs(k.double().cpu().numpy() - wk) <= 2.0 ** -4 * (np.abs(wk) + rk) + 2.0 ** -10 * s + rk)
        # the scale fits what stands there, unless a border is nearer than the rotation's error
        for p in sorted(set((slots // page).tolist())):
            top = np.abs(wk[slots // page == p]).max((0, 2))
            old = before[0].scale[p] if p == slots[0] // page else np.zeros(n_kv)
            got = cache.k_scale[p].double().cpu().numpy()
            for h in range(n_kv):
                assert got[h] in (max(_need(top[h] * (1 - 1e-5)), old[h]), max(_need(top[h] * (1 + 1e-5)), old[h]))
        before[1].write(slots, x[:, n_q + n_kv:])
        sv = cache.v_scale.double().cpu().numpy()
        assert np.array_equal(sv, before[1].scale)
        want_v = _values(before[1].codes[slots // page, :, slots % page]) * sv[slots // page][:, :, None]
        assert np.array_equal(v.double().cpu().numpy(), want_v)


def test_rows_without_a_position_and_q_in_place(env):
    torch, kvd = env
    cache = _cache(torch, kvd, 4, 16, 2, 64)
    x = torch.randn(20, 8, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).bfloat16()
    pos, slots = list(range(17)) + [-1, -2, -1], list(range(17)) + [-1, -1, -1]
    plan, table = _plan(torch, kvd, pos, slots), kvd.RopeTable(64)
    want = kvd.paged_append(cache, plan, x[:, 4:6], x[:, 6:], q=x[:, :4], rope=table)
    y = x.clone()
    again = _cache(torch, kvd, 4, 16, 2, 64)
    assert kvd.paged_append(again, plan, y[:, 4:6], y[:, 6:], q=y[:, :4], q_out=y[:, :4], rope=table).data_ptr() == y.data_ptr()
    assert torch.equal(y[:17, :4], want[:17]) and torch.equal(y[17:], x[17:]) and torch.equal(y[:, 4:], x[:, 4:])
    assert torch.equal(again.k.view(torch.uint8), cache.k.view(torch.uint8)) and torch.equal(again.k_scale, cache.k_scale)
    assert kvd.paged_append(cache, plan, x[:, 4:6].float(), x[:, 6:].float(), q=x[:, :4].float()).dtype is torch.bfloat16


# ---------------------------------------------------------------- reading back


@pytest.mark.parametrize("pages", ["e4m3", "f16", "bf16"])
@pytest.mark.parametrize("to", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hd,page,n_kv", [(128, 16, 3), (64, 128, 2), (128, 64, 8)])
def test_read_gives_rows_back(env, pages, to, hd, page, n_kv):
    torch, kvd = env
    lens = [0, 1, page, page + 1, 3 * page - 1, 517, 40]
    start = [0, 0, 3, page, 1, 100, 40]
    n = [0, 1, page - 3, 1, 3 * page - 2, 300, 0]
    if pages == "e4m3":
        cache, rows = _poisoned8(torch, kvd, lens, n_kv, hd, page, 5)
    else:
        from test_gpu_paged import _poisoned
        cache, rows = _poisoned(torch, kvd, lens, n_kv, hd, page, _dt(torch, pages), 5)
    dt, total = _dt(torch, to), sum(n)
    box = torch.full((2, total + 4, n_kv, hd + 16), 9.0, device="cuda", dtype=dt)  # rows with room behind them
    k_out, v_out = box[0, ..., :hd], box[1, ..., :hd]
    cu = _i32(torch, [0] + np.cumsum(n).tolist())
    assert kvd.paged_read(cache, cu, total + 4, start=_i32(torch, start), k_out=k_out, v_out=v_out)[0] is k_out
    assert cache.device_error() == 0 and bool((box[:, total:] == 9).all()) and bool((box[..., hd:] == 9).all())
    at = 0
    for b, m in enumerate(n):
        for got, want in zip((k_out, v_out), rows[b]):
            assert torch.equal(got[at:at + m], want[start[b]:start[b] + m].to(dt))
        at += m
    whole = kvd.paged_read(cache, _i32(torch, [0] + np.cumsum(lens).tolist()), sum(lens), dtype=dt)
    for i in range(2):
        assert torch.equal(whole[i], torch.cat([r[i] for r in rows]).to(dt))
    assert cache.device_error() == 0


def test_read_beyond_what_is_held(env):
    torch, kvd = env
    cache, rows = _poisoned8(torch, kvd, [20, 5, 40], 2, 64, 16, 6)
    cache.block_table[2, 1] = cache.n_pages
    k, v = kvd.paged_read(cache, _i32(torch, [0, 25, 30, 70]), 70, dtype=torch.float32)
    assert cache.device_error() == 2
    assert torch.equal(k[:20], rows[0][0].float()) and not k[20:25].any() and not v[46:62].any()
    assert torch.equal(k[25:30], rows[1][0].float()) and torch.equal(v[62:], rows[2][1][32:].float())
    for start in ([-1, 0, 0], [2 ** 31 - 1, 0, 0]):
        k, _ = kvd.paged_read(cache, _i32(torch, [0, 1, 1, 1]), 1, start=_i32(torch, start), dtype=torch.float32)
        assert cache.device_error() == 2 and not k.any()
    cache.k_scale.fill_(math.nan)
    k, v = kvd.paged_read(cache, _i32(torch, [0, 20, 20, 20]), 20, dtype=torch.float32)
    assert cache.device_error() == 2 and torch.equal(v, rows[0][1].float()) and not bool(torch.isnan(k).any())
    out = torch.full((3, 2, 64), 4.0, device="cuda")
    kvd.paged_read(cache, _i32(torch, [0, 0, 0, 0]), 3, k_out=out, v_out=out.clone())
    assert bool((out == 4).all())
    assert kvd.paged_read(cache, _i32(torch, [0, 0, 0, 0]), 0)[0].shape == (0, 2, 64)


# ---------------------------------------------------------------- attention


def _poisoned8(torch, kvd, lens, n_kv, hd, page, seed, spare=3, spread=2.0, odd_scales=False):
    """Pages of random codes for requests of these lengths, shuffled, with NaN in every row that no request holds, nonsense in the
    table's unused places and in the scales of free pages; the rows (f64) of each request beside it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    has = [-(-n // page) for n in lens]
    n_pages = sum(has) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    width = max(has) + 2
    codes = [torch.full((n_pages, n_kv, page, hd), 0x7f, device="cuda", dtype=torch.uint8) for _ in range(2)]
    scales = [torch.full((n_pages, n_kv), float("nan"), device="cuda") for _ in range(2)]
    table = torch.tensor([[2 ** 31 - 1, -7, n_pages][i % 3] for i in range(len(lens) * width)], dtype=torch.int32).view(len(lens), width)
    rows = []
    for b, n in enumerate(lens):
        pair = []
        pages = [order.pop() for _ in range(has[b])]
        table[b, : has[b]] = torch.tensor(pages, dtype=torch.int32)
        for c, s in zip(codes, scales):
            x = torch.randn(n, n_kv, hd, generator=g, device="cuda")
            size = torch.exp2((torch.rand(has[b], n_kv, generator=g, device="cuda") - 0.5) * spread) / 64
            if not odd_scales:
                size = torch.exp2(torch.floor(torch.log2(size)))
            per_row = size.repeat_interleave(page, 0)[:n, :, None]
            y = (x / per_row).clamp(-448, 448).to(torch.float8_e4m3fn)
            pair.append(y.double() * per_row.double())
            for i, p in enumerate(pages):
                part = slice(i * page, min(n, (i + 1) * page))
                c[p, :, : part.stop - part.start] = y[part].view(torch.uint8).transpose(0, 1)
                s[p] = size[i]
        rows.append(tuple(pair))
    k, v = (c.view(torch.float8_e4m3fn) for c in codes)
    return kvd.PagedKvCache.of(k, v, table.cuda(), _i32(torch, lens), k_scale=scales[0], v_scale=scales[1]), rows


def _attend8(torch, q, k, v, total, scale, window=0, softcap=0.0, sink=None):
    """64-bit attention; returns out and its tolerance but for the type's rounding, as the 16-bit pages' reference does, with q's."""
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
        x, kk, vv = q[:, h].double(), k[:, h // grp], v[:, h // grp]
        s = x @ kk.T * scale
        d = hd * 2.0 ** -24 * scale * (x.abs() @ kk.abs().T) + 2.0 ** -17 * scale * x.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[None]
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


def _check8(torch, got, ref, v_top):
    """_check_attend with what a weight's range takes: 128 * 2^-22 * 448 * the largest scale of V."""
    out, size, slack = ref
    half = float(torch.finfo(got.dtype).eps) / 2
    tol = (half + slack * (1 + half)) * size * (1 + half) + half * out.abs() + _tiny(torch, got.dtype) + 2.0 ** -15 * 448 * v_top
    d = (got.double() - out).abs()
    assert not bool(torch.isnan(got).any())
    assert bool((d <= tol).all()), float((d / tol).max())
    # and a mean over all: roundings are as often up as down
    assert float((d ** 2).mean().sqrt()) <= 2 * half * float((size ** 2).mean().sqrt()) + 2.0 ** -15 * v_top * 8 + float(slack.max()) * float(size.max())


def _run8(torch, kvd, lens, new, n_kv, group, hd, page, dt, seed, window=0, softcap=0.0, sinks=False, scale=None, tail=3, sample=None, **pages):
    cache, rows = _poisoned8(torch, kvd, lens, n_kv, hd, page, seed, **pages)
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
    v_top = float(cache.v_scale.nan_to_num(0).max())
    for b, n in enumerate(new):
        if n and (sample is None or b in sample):
            kk, vv = rows[b]
            live = min(n, lens[b])  # a position below zero sees nothing
            assert not out[at:at + n - live].any()
            if live:
                want = _attend8(torch, q[at + n - live:at + n], kk, vv, lens[b], scale, window, softcap, sink)
                _check8(torch, out[at + n - live:at + n], want, v_top)
        at += n
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,page", [(1, 16), (4, 64), (16, 128), (5, 32)])
def test_attention_of_single_tokens(env, dtype, hd, group, page):
    torch, kvd = env
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700, 0, 2049]
    _run8(torch, kvd, lens, [1 if n else 0 for n in lens], 2, group, hd, page, _dt(torch, dtype), group)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,page", [(1, 128), (2, 16), (3, 32), (8, 64), (16, 16)])
def test_attention_of_chunks(env, dtype, hd, group, page):
    """Chunks around the tiles' edges."""
    torch, kvd = env
    tile = 128 // group
    new = [1, tile - 1 or 1, tile, tile + 1, 2 * tile, 2 * tile + 1, 0, 4 * tile + 3, 3 * tile, 7]
    lens = [n + x for n, x in zip(new, [0, 5, 128 - tile if tile < 128 else 0, 300, 0, 77, 9, 1000, 129, 1500])]
    _run8(torch, kvd, lens, new, 2, group, hd, page, _dt(torch, dtype), 100 + group)


@pytest.mark.parametrize("hd,group", [(64, 2), (128, 4), (128, 1)])
@pytest.mark.parametrize("window,softcap,sinks", [(1, 0.0, False), (2, 0.0, True), (100, 0.0, False), (128, 30.0, False), (1000, 5.0, True), (0, 30.0, False),
                                                  (0, 0.0, True), (1 << 40, 0.0, False)])
def test_attention_options(env, hd, group, window, softcap, sinks):
    torch, kvd = env
    for dt in (torch.bfloat16, torch.float16):
        _run8(torch, kvd, [900, 1, 130, 2000, 64], [1, 1, 130, 300, 3], 2, group, hd, 16, dt, 7, window, softcap, sinks)


@pytest.mark.parametrize("drafts,group", [(2, 8), (4, 4), (5, 4), (4, 16), (8, 8), (9, 8), (33, 1), (3, 5)])
def test_attention_of_drafts(env, drafts, group):
    """A few rows for each request: 16, 32, 64 query rows a KV head and one more."""
    torch, kvd = env
    for dt, hd in ((torch.bfloat16, 128), (torch.float16, 64), (torch.float16, 128)):
        _run8(torch, kvd, [drafts, 700, 129, 4001], [drafts, drafts, max(drafts - 1, 1), drafts], 2, group, hd, 32, dt, drafts)


def test_attention_rows_that_see_nothing_are_zero(env):
    torch, kvd = env
    for sinks in (False, True):
        _run8(torch, kvd, [3, 0, 130, 0], [5, 2, 400, 1], 2, 4, 128, 16, torch.bfloat16, 11, sinks=sinks)


def test_attention_cuts_long_requests(env):
    torch, kvd = env
    for dt, hd in ((torch.bfloat16, 128), (torch.float16, 64)):
        _run8(torch, kvd, [60001], [1], 1, 8, hd, 64, dt, 21)
        _run8(torch, kvd, [30011, 5, 900], [3, 5, 1], 2, 4, hd, 16, dt, 22, sinks=True)
        _run8(torch, kvd, [9000], [700], 1, 4, hd, 128, dt, 23, softcap=20.0, sinks=True)
        _run8(torch, kvd, [20000], [130], 1, 1, hd, 32, dt, 24, window=5000)


def test_attention_of_many_requests(env):
    torch, kvd = env
    r = np.random.default_rng(2)
    lens = r.integers(0, 40, 1100).tolist()
    new = [int(r.integers(0, min(n, 3) + 1)) for n in lens]
    _run8(torch, kvd, lens, new, 1, 2, 64, 16, torch.bfloat16, 31, sample=set(range(0, 1100, 13)) | {0, 1, 1098, 1099})
    assert _run8(torch, kvd, [5, 7], [0, 0], 1, 2, 64, 16, torch.bfloat16, 31).shape[0] == 3


@pytest.mark.parametrize("seed", range(10))
def test_attention_of_mixed_batches(env, seed):
    """Prompts, drafts, single tokens, requests without new rows and without rows, in any order and length."""
    torch, kvd = env
    r = np.random.default_rng(100 + seed)
    n = int(r.integers(3, 24))
    lens = [int(x) for x in np.exp(r.uniform(0, math.log(2500), n)).astype(int)]
    new = [min(x, int(r.choice([0, 1, 1, 1, 4, 17, 64, 130, 300]))) for x in lens]
    group, hd, page = int(r.choice([1, 2, 3, 4, 8, 16])), int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128]))
    _run8(torch, kvd, lens, new, int(r.integers(1, 4)), group, hd, page, [torch.bfloat16, torch.float16][seed % 2], 300 + seed,
          window=int(r.choice([0, 0, 77, 600])), softcap=float(r.choice([0.0, 0.0, 20.0])), sinks=bool(r.integers(0, 2)))


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("spread", [0.0, 6.0, 16.0])
def test_attention_over_scales_of_any_size(env, spread, odd):
    """Blocks whose scales lie far apart inside one tile, powers of two or not."""
    torch, kvd = env
    for dt, hd, new in ((torch.bfloat16, 128, 1), (torch.float16, 64, 1), (torch.bfloat16, 64, 200), (torch.float16, 128, 140)):
        _run8(torch, kvd, [900, 333], [new, new], 2, 4, hd, 16, dt, 41, spread=spread, odd_scales=odd, scale=0.02)


@pytest.mark.parametrize("scale", [1e-4, 0.05, 3.0])
def test_attention_of_flat_and_sharp_softmaxes(env, scale):
    torch, kvd = env
    for dt in (torch.bfloat16, torch.float16):
        _run8(torch, kvd, [3000, 700], [1, 200], 2, 4, 128, 16, dt, 51, scale=scale)


def test_many_small_weights_beside_a_large_one(env):
    """One row that takes most of the weight and thousands that share the rest: none of them may be lost."""
    torch, kvd = env
    hd, page, total = 128, 64, 40000
    for dt in (torch.bfloat16, torch.float16):
        for new in (1, 150):
            k = torch.zeros(total, 1, hd, device="cuda")
            k[0, 0, 0] = 1.0
            v = torch.full((total, 1, hd), 1.0, device="cuda")
            v[0] = -1.0
            cache = kvd.PagedKvCache(total // page + 1, page, 1, hd, 1, total // page + 1, dtype=torch.float8_e4m3fn)
            cache.block_table.copy_(torch.arange(total // page + 1, dtype=torch.int32)[None])
            cache.seq_len.fill_(total)
            kvd.paged_append(cache, _plan(torch, kvd, range(total), range(total)), k, v)
            q = torch.zeros(new, 2, hd, device="cuda", dtype=dt)
            q[..., 0] = 10.0
            plan = kvd.PagedPlan(_i32(torch, [0, new]), cache.seq_len)
            out = kvd.paged_attention(q, cache, plan, scale=1.0).double()
            n = torch.arange(total - new + 1, total + 1, device="cuda").double()[:, None, None] - 1
            want = (n - math.exp(10)) / (n + math.exp(10))
            # weights exp(-10) = 4.5e-5 of the largest, rounded to q's type: a bias of half a step at most
            half = float(torch.finfo(dt).eps) / 2
            assert float((out - want).abs().max()) <= half * (1 + 1) + 2.0 ** -14


def test_attention_with_growing_scores(env):
    """Keys that grow along the request: the maximum moves in every tile."""
    torch, kvd = env
    hd, page, total = 128, 16, 1500
    g = torch.Generator(device="cuda").manual_seed(9)
    cache, rows = _poisoned8(torch, kvd, [total], 1, hd, page, 61)
    grow = torch.exp2(torch.arange(-(-total // page), device="cuda") / 12 - 8).floor_divide(2.0 ** -30) * 2.0 ** -30
    for i in range(-(-total // page)):
        cache.k_scale[cache.block_table[0, i].long()] *= grow[i]
    kk = rows[0][0] * grow.double().repeat_interleave(page)[:total, None, None]
    for dt in (torch.bfloat16, torch.float16):
        q = torch.randn(131, 4, hd, generator=g, device="cuda").to(dt)
        for new in (1, 131):
            plan = kvd.PagedPlan(_i32(torch, [0, new]), cache.seq_len)
            out = kvd.paged_attention(q[:new], cache, plan, scale=0.05)
            _check8(torch, out, _attend8(torch, q[:new], kk, rows[0][1], total, 0.05), float(cache.v_scale.nan_to_num(0).max()))


def test_attention_takes_views_and_queries_of_any_size(env):
    torch, kvd = env
    cache, rows = _poisoned8(torch, kvd, [300, 40], 2, 128, 16, 71)
    g = torch.Generator(device="cuda").manual_seed(1)
    v_top = float(cache.v_scale.nan_to_num(0).max())
    plan = kvd.PagedPlan(_i32(torch, [0, 2, 42]), cache.seq_len)
    wide = torch.randn(42, 12, 128, generator=g, device="cuda").bfloat16()
    q = wide[:, 2:10]
    out = torch.zeros(8, 42, 128, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    kvd.paged_attention(q, cache, plan, out=out)
    for a, e, b in ((0, 2, 0), (2, 42, 1)):
        _check8(torch, out[a:e], _attend8(torch, q[a:e], *rows[b], [300, 40][b], 128 ** -0.5), v_top)
    # rows of zeros, and rows whose size lies far from one
    for size in (0.0, 1e-30, 1e30):
        y = (q.float() * size).bfloat16()
        got = kvd.paged_attention(y, cache, plan, scale=128 ** -0.5 / (size or 1.0))
        for a, e, b in ((0, 2, 0), (2, 42, 1)):
            _check8(torch, got[a:e], _attend8(torch, y[a:e], *rows[b], [300, 40][b], 128 ** -0.5 / (size or 1.0)), v_top)


def test_attention_skips_malformed_requests(env):
    torch, kvd = env
    lens = [100, 9, 70, 300]
    cache, rows = _poisoned8(torch, kvd, lens, 1, 64, 16, 81)
    cu = [0, 2, 3, 7, 8]
    q = torch.randn(8, 4, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    wide, v_top = cache.block_table.shape[1] * 16, float(cache.v_scale.nan_to_num(0).max())
    for bad_len in (-1, wide + 1, 2 ** 31 - 1):
        out = torch.full_like(q, 5.0)
        kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, cu), _i32(torch, [100, bad_len, 70, 300])), out=out)
        assert cache.device_error() == 2 and bool((out[2] == 5).all())
        for a, e, b in ((0, 2, 0), (3, 7, 2), (7, 8, 3)):
            _check8(torch, out[a:e], _attend8(torch, q[a:e], *rows[b], lens[b], 1 / 8), v_top)
    for bad_cu in ([0, 2, 1, 7, 8], [0, 2, 3, 7, 9], [-1, 2, 3, 7, 8]):
        kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, bad_cu), cache.seq_len))
        assert cache.device_error() == 2
    # a scale that cannot be one is the block's alone
    keep = cache.k_scale.clone()
    cache.k_scale[cache.block_table[3, 2].long()] = math.nan
    out = kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, cu), cache.seq_len))
    assert cache.device_error() == 2 and not bool(torch.isnan(out).any())
    for a, e, b in ((0, 2, 0), (2, 3, 1), (3, 7, 2)):
        _check8(torch, out[a:e], _attend8(torch, q[a:e], *rows[b], lens[b], 1 / 8), v_top)
    cache.k_scale.copy_(keep)
    cache.block_table[3, 2] = cache.n_pages
    out = kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, cu), cache.seq_len))
    assert cache.device_error() == 2 and not bool(torch.isnan(out).any())
    for a, e, b in ((0, 2, 0), (2, 3, 1), (3, 7, 2)):
        _check8(torch, out[a:e], _attend8(torch, q[a:e], *rows[b], lens[b], 1 / 8), v_top)


# ---------------------------------------------------------------- together


STEPS = [([40, 7, 0, 200], None), ([1, 1, 1, 1], None), ([1, 4, 130, 1], None), ([1, 1, 1, 0], [41, 0, 131, 60]), ([3, 300, 1, 90], [0, 1, 132, 60]),
         ([0, 1, 1, 1], None), ([1, 1, 0, 5], [3, 301, 0, 145])]


def _step(kvd, cache, new, keep, room, x, n_q, n_kv, table, plan=None, ws=None):
    plan = kvd.paged_plan(cache, new, room, keep_len=keep, plan=plan)
    q = kvd.paged_append(cache, plan, x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:], q=x[:, :n_q], rope=table)
    return plan, q, kvd.paged_attention(q, cache, plan, workspace=ws)


@pytest.mark.parametrize("dtype,hd,group,page", [("bf16", 128, 4, 16), ("f16", 64, 2, 64), ("f32", 128, 16, 128)])
def test_a_server_runs_steps_over_8_bits(env, dtype, hd, group, page):
    """Prompts, decode steps, drafts rejected, requests dropped and started again in one batch; what is attended is what is read back, and
    what is read back stays near what was written."""
    torch, kvd = env
    n_kv, n_seq = 2, 4
    n_q = n_kv * group
    cache = kvd.PagedKvCache(800 // page + 8, page, n_kv, hd, n_seq, 400 // page + 2, dtype=torch.float8_e4m3fn)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x7f)
    held = [np.zeros((0, n_kv, hd)) for _ in range(n_seq)]
    table, now = kvd.RopeTable(hd, "half"), [0] * n_seq
    for i, (new, keep) in enumerate(STEPS):
        room = max(sum(new) + (i % 3) * 5, 1)
        g = torch.Generator(device="cuda").manual_seed(100 + i)
        x = (torch.randn(room, n_q + 2 * n_kv, hd, generator=g, device="cuda") * 2.0 ** (i % 4)).to(_dt(torch, dtype))
        x[:, :n_q] *= 2.0 ** -(i % 4)
        plan, q, out = _step(kvd, cache, _i32(torch, new), None if keep is None else _i32(torch, keep), room, x, n_q, n_kv, table)
        assert cache.device_error() == 0, i
        now = [a + n for a, n in zip(now if keep is None else keep, new)]
        assert cache.seq_len.tolist() == now
        k, v = kvd.paged_read(cache, _i32(torch, [0] + np.cumsum(now).tolist()), sum(now), dtype=torch.float32)
        at = row = 0
        for b, n in enumerate(new):
            kk, vv = k[row:row + now[b]].double(), v[row:row + now[b]].double()
            if n:
                want = _attend8(torch, q[at:at + n], kk, vv, now[b], hd ** -0.5)
                _check8(torch, out[at:at + n], want, float(cache.v_scale.max()))
            given = x[at:at + n, n_q + n_kv:].double().cpu().numpy()
            held[b] = np.concatenate([held[b][: now[b] - n], given])
            # half a step of each value, twice where a subnormal moved to a larger scale, of which 16 is the largest here
            worst = np.abs(vv.cpu().numpy() - held[b])
            assert np.all(worst <= 2.0 ** -4 * np.abs(held[b]) + 2 * 2.0 ** -10 * float(cache.v_scale.max()))
            at, row = at + n, row + now[b]


def test_a_captured_step_replays(env):
    """One graph of plan, append, attention and read, replayed with new numbers, against the same steps run eagerly."""
    torch, kvd = env
    room, hd, n_kv, n_q, page = 420, 128, 2, 8, 16
    def make():
        c = kvd.PagedKvCache(60, page, n_kv, hd, 4, 27, dtype=torch.float8_e4m3fn)
        c.k.view(torch.uint8).fill_(0x7f)
        c.v.view(torch.uint8).fill_(0x7f)
        return c
    eager, replayed = make(), make()
    new, keep, cu = _i32(torch, [0] * 4), _i32(torch, [0] * 4), _i32(torch, [0] * 5)
    x = torch.randn(room, n_q + 2 * n_kv, hd, device="cuda").bfloat16()
    table = kvd.RopeTable(hd, "half")
    rows = torch.zeros(2, 900, n_kv, hd, device="cuda")
    for _ in range(2):
        plan, _, _ = _step(kvd, replayed, new, keep, room, x, n_q, n_kv, table)
        kvd.paged_read(replayed, cu, 900, k_out=rows[0], v_out=rows[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan, q, out = _step(kvd, replayed, new, keep, room, x, n_q, n_kv, table, plan=plan)
        kvd.paged_read(replayed, cu, 900, k_out=rows[0], v_out=rows[1])
    now = [0] * 4
    for i, (n, k) in enumerate(STEPS):
        k = list(now) if k is None else k
        now = [a + b for a, b in zip(k, n)]
        gen = torch.Generator(device="cuda").manual_seed(200 + i)
        x.copy_(torch.randn(room, n_q + 2 * n_kv, hd, generator=gen, device="cuda"))
        new.copy_(_i32(torch, n))
        keep.copy_(_i32(torch, k))
        cu.copy_(_i32(torch, [0] + np.cumsum(now).tolist()))
        out.fill_(2.0)
        g.replay()
        _, _, want = _step(kvd, eager, _i32(torch, n), _i32(torch, k), room, x, n_q, n_kv, table)
        t = sum(n)
        assert torch.equal(out[:t], want[:t]) and bool((out[t:] == 2).all()), i
        back = kvd.paged_read(eager, cu, sum(now), dtype=torch.float32)
        assert torch.equal(rows[0, : sum(now)], back[0]) and torch.equal(rows[1, : sum(now)], back[1])
        assert torch.equal(replayed.k.view(torch.uint8), eager.k.view(torch.uint8)) and replayed.device_error() == 0 and eager.device_error() == 0


def test_two_streams_repeats_and_another_stream(env):
    """Calls on two streams at once, repeats and outputs made for another stream give the same bits."""
    torch, kvd = env
    pairs = []
    for seed, lens, new in ((1, [5000, 30, 900], [1, 1, 4]), (2, [2000, 700], [300, 1])):
        cache, _ = _poisoned8(torch, kvd, lens, 2, 128, 32, seed)
        q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).bfloat16()
        plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
        pairs.append((cache, q, plan, kvd.paged_attention(q, cache, plan)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(20):
        outs = [kvd.paged_attention(q, c, p, stream=s) for (c, q, p, _), s in zip(pairs, streams)]
        reads = [kvd.paged_read(c, _i32(torch, [0, 30] + [30] * (c.n_seq - 1)), 30, stream=s) for (c, q, p, _), s in zip(pairs, streams)]
        torch.cuda.synchronize()
        for o, r, (c, _, _, want) in zip(outs, reads, pairs):
            assert torch.equal(o, want)
            assert torch.equal(r[0], kvd.paged_read(c, _i32(torch, [0, 30] + [30] * (c.n_seq - 1)), 30)[0])


def test_rows_read_back_feed_the_contiguous_cache(env):
    """A request leaves the pages: its rows, read back in f32, are appended to a layer cache, whose decode gives the same attention."""
    torch, kvd = env
    cache, rows = _poisoned8(torch, kvd, [500], 2, 128, 16, 91)
    k, v = kvd.paged_read(cache, _i32(torch, [0, 500]), 500, dtype=torch.float32)
    layer = kvd.LayerKvCache(1, 2, 128, "f32", 512)
    kvd.kv_append(layer, k, v, [500])
    q = torch.randn(1, 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).half()
    flat = kvd.decode_attention(q.float(), layer, scale=128 ** -0.5)
    paged = kvd.paged_attention(q, cache, kvd.PagedPlan(_i32(torch, [0, 1]), cache.seq_len))
    want = _attend8(torch, q, *rows[0], 500, 128 ** -0.5)
    _check8(torch, paged, want, float(cache.v_scale.nan_to_num(0).max()))
    assert float((flat.double() - want[0]).abs().max()) <= 2e-5 * float(want[0].square().mean().sqrt())


def test_layers_share_tables(env):
    torch, kvd = env
    a = kvd.PagedKvCache(8, 16, 2, 64, 2, 4, dtype=torch.float8_e4m3fn)
    b = a.layer_like()
    assert b.k.dtype is torch.float8_e4m3fn and b.k_scale.shape == (8, 2) and b.k_scale.data_ptr() != a.k_scale.data_ptr()
    assert b.block_table is a.block_table and b.error is a.error


def test_a_failed_launch_is_reported(env):
    torch, kvd = env
    from kv_cache_decode_attention_gb300 import _abi

    cache, _ = _poisoned8(torch, kvd, [300], 2, 64, 16, 3)
    q = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    plan = kvd.PagedPlan(_i32(torch, [0, 1]), cache.seq_len, None, _i32(torch, [299]), _i32(torch, [3]))
    calls = (lambda: kvd.paged_attention(q, cache, plan), lambda: kvd.paged_append(cache, plan, q[:, :2], q[:, 2:]),
             lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 1))
    for call in calls:
        _abi.call("kvd_test_fail_after", 0)
        with pytest.raises(kvd.KvdError) as e:
            call()
        assert e.value.status == _abi.ECUDA
        call()
    torch.cuda.synchronize()


def test_python_checks_of_8_bits(env):
    torch, kvd = env
    cache, _ = _poisoned8(torch, kvd, [300], 2, 64, 16, 3)
    q = torch.zeros(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    plan = kvd.PagedPlan(_i32(torch, [0, 1]), cache.seq_len, None, _i32(torch, [299]), _i32(torch, [3]))
    of = lambda **kw: kvd.PagedKvCache.of(**{**dict(k=cache.k, v=cache.v, block_table=cache.block_table, seq_len=cache.seq_len, k_scale=cache.k_scale,  # noqa: E731
                                                    v_scale=cache.v_scale), **kw})
    of()
    for bad in (lambda: of(k_scale=None), lambda: of(v_scale=None), lambda: of(k_scale=cache.k_scale[:-1]), lambda: of(v_scale=cache.v_scale.double()),
                lambda: of(k_scale=cache.k_scale.cpu()), lambda: of(v_scale=cache.v_scale.t().contiguous().t()), lambda: of(k=cache.k.bfloat16()),
                lambda: of(k=cache.k.bfloat16(), v=cache.v.bfloat16()), lambda: of(k=cache.k.view(torch.float8_e5m2), v=cache.v.view(torch.float8_e5m2)),
                lambda: of(k=None, v=None, page_size=16, free_pages=cache.seq_len, n_free=cache.error),
                lambda: kvd.paged_attention(q.float(), cache, plan), lambda: kvd.paged_attention(q.to(torch.float8_e4m3fn), cache, plan),
                lambda: kvd.paged_attention(q, cache, plan, out=q.half()), lambda: kvd.paged_attention(q[..., :32], cache, plan),
                lambda: kvd.paged_append(cache, plan, q[:, :2], q[:, 2:].half()), lambda: kvd.paged_append(cache, plan, q[:, :2], q[:, 2:], q=q, q_out=q.half()),
                lambda: kvd.paged_append(cache, plan, q[:, :2].float(), q[:, 2:].float(), q=q.float(), q_out=q.float()),
                lambda: kvd.paged_append(cache, plan, q[:, :2].float(), q[:, 2:].float(), q=q.float(), q_out=q.to(torch.float8_e4m3fn)),
                lambda: kvd.paged_append(cache, plan, q[:, :2].double(), q[:, 2:].double()),
                lambda: kvd.paged_read(cache, _i32(torch, [0, 1, 2]), 1), lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), -1),
                lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 1, dtype=torch.float64), lambda: kvd.paged_read(cache, _i32(torch, [0, 1]).long(), 1),
                lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 1, start=_i32(torch, [0, 0])),
                lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 1, k_out=q[:, :2], v_out=q[:, 2:].half()),
                lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 2, k_out=q[:, :2]), lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 1, k_out=q[0])):
        with pytest.raises(ValueError):
            bad()
    # outputs that share memory
    for bad in (lambda: kvd.paged_attention(q, cache, plan, out=q), lambda: kvd.paged_read(cache, _i32(torch, [0, 1]), 1, k_out=q[:, :2], v_out=q[:, 1:3]),
                lambda: kvd.paged_append(cache, plan, cache.k.view(torch.bfloat16).view(-1)[:128].view(1, 2, 64), q[:, 2:]),
                lambda: kvd.paged_append(of(v=cache.k), plan, q[:, :2], q[:, 2:]), lambda: kvd.paged_append(of(v_scale=cache.k_scale), plan, q[:, :2], q[:, 2:])):
        with pytest.raises(kvd.KvdError):
            bad()


def test_a_pool_past_31_bits_of_bytes(env):
    """Codes past 2^31 and 2^32 bytes from the pool's start."""
    torch, kvd = env
    n_pages, page, n_kv, hd = 36000, 128, 8, 128  # 4.7 GB of K
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    cache = kvd.PagedKvCache(n_pages, page, n_kv, hd, 1, 8, dtype=torch.float8_e4m3fn)
    cache.block_table[0, :3] = _i32(torch, [n_pages - 1, 18000, 3])
    cache.seq_len.fill_(300)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(300, 3 * n_kv, hd, generator=g, device="cuda").bfloat16()
    pos = np.arange(300)
    slots = np.array([n_pages - 1, 18000, 3])[pos // page] * page + pos % page
    kvd.paged_append(cache, _plan(torch, kvd, pos, slots), x[:, n_kv:2 * n_kv], x[:, 2 * n_kv:])
    k, v = kvd.paged_read(cache, _i32(torch, [0, 300]), 300, dtype=torch.float32)
    assert float((v - x[:, 2 * n_kv:].float()).abs().max()) <= 2.0 ** -4 * 6
    plan = kvd.PagedPlan(_i32(torch, [0, 2]), cache.seq_len)
    out = kvd.paged_attention(x[:2, :n_kv], cache, plan)
    assert cache.device_error() == 0
    _check8(torch, out, _attend8(torch, x[:2, :n_kv], k.double(), v.double(), 300, hd ** -0.5), float(cache.v_scale.max()))


@pytest.mark.parametrize("lens,new", [([30000], [1]), ([5000, 30, 900, 3000], [1, 1, 4, 1]), ([4000, 1500, 700], [300, 1, 90])])
def test_a_launch_given_up_leaves_no_trace(env, lens, new):
    """One block's waits end early, at one moment or another: the error bit, and the next calls and replays right."""
    torch, kvd = env
    from kv_cache_decode_attention_gb300 import _abi

    cache, _ = _poisoned8(torch, kvd, lens, 2, 128, 16, 3)
    q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
    ws = torch.zeros(kvd.paged_attention_workspace(sum(new), 8, 2, 128, torch.float8_e4m3fn), dtype=torch.uint8, device="cuda")
    want, out = kvd.paged_attention(q, cache, plan, workspace=ws), torch.empty_like(q)
    assert cache.device_error() == 0
    gave_up = 0
    try:
        for cta in (0, 37, 76, 151):
            for after in (0, 2000, 5000, 9000):
                assert _abi.lib().kvd_test_give_up(cta, after) == 0
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    kvd.paged_attention(q, cache, plan, out=out, workspace=ws)
                _abi.lib().kvd_test_give_up(-1, 0)
                for _ in range(3):
                    out.fill_(float("nan"))
                    graph.replay()
                    error = cache.device_error()
                    assert error in (0, 1)
                    gave_up += error
                    assert error == 1 or torch.equal(out, want)
                assert torch.equal(kvd.paged_attention(q, cache, plan, out=out, workspace=ws), want) and cache.device_error() == 0
    finally:
        _abi.lib().kvd_test_give_up(-1, 0)
    assert gave_up >= 3


def _banded(torch, shape, dtype, fill):
    """A contiguous tensor between two bands of 4 KB, and what tells whether they stand."""
    size = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    room = -(-size // 256) * 256
    box = torch.full((8192 + room,), 0x5a, dtype=torch.uint8, device="cuda")
    inner = box[4096:4096 + size].view(dtype).view(shape)
    inner.fill_(fill)
    return inner, lambda: bool((box[:4096] == 0x5a).all()) and bool((box[4096 + size:] == 0x5a).all())


@pytest.mark.parametrize("hd,group,dtype", [(128, 4, "bf16"), (64, 16, "f16"), (128, 1, "f16")])
def test_nothing_is_written_beside_the_outputs(env, hd, group, dtype):
    """Workspace of exactly the size that is asked for, outputs, codes and scales between guard bands."""
    torch, kvd = env
    n_kv, page, dt = 2, 16, _dt(torch, dtype)
    for lens, new in (([9000, 40], [1, 1]), ([600, 3000, 20], [130, 7, 20])):
        src, rows = _poisoned8(torch, kvd, lens, n_kv, hd, page, 7)
        t = sum(new)
        q = torch.randn(t, n_kv * group, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dt)
        plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), src.seq_len)
        out, ok_out = _banded(torch, q.shape, dt, 0)
        ws, ok_ws = _banded(torch, (kvd.paged_attention_workspace(t, n_kv * group, n_kv, hd, torch.float8_e4m3fn),), torch.uint8, 0xff)
        kvd.paged_attention(q, src, plan, out=out, workspace=ws)
        assert torch.equal(out, kvd.paged_attention(q, src, plan)) and ok_out() and ok_ws()
        k_out, ok_k = _banded(torch, (sum(lens), n_kv, hd), torch.float32, 0)
        v_out, ok_v = _banded(torch, (sum(lens), n_kv, hd), torch.float32, 0)
        kvd.paged_read(src, _i32(torch, [0] + np.cumsum(lens).tolist()), sum(lens), k_out=k_out, v_out=v_out)
        assert ok_k() and ok_v() and torch.equal(k_out, torch.cat([r[0] for r in rows]).float())
        parts = [_banded(torch, (5, n_kv, page, hd), torch.uint8, 0) for _ in range(2)] + [_banded(torch, (5, n_kv), torch.float32, 1) for _ in range(2)]
        cache = kvd.PagedKvCache.of(parts[0][0].view(torch.float8_e4m3fn), parts[1][0].view(torch.float8_e4m3fn), _i32(torch, [[0, 1, 2, 3, 4]]), _i32(torch, [80]),
                                    k_scale=parts[2][0], v_scale=parts[3][0])
        x = torch.randn(80, 2 * n_kv, hd, device="cuda")
        q_out, ok_q = _banded(torch, (80, n_kv, hd), torch.bfloat16, 0)
        kvd.paged_append(cache, _plan(torch, kvd, range(80), range(80)), x[:, :n_kv], x[:, n_kv:], q=x[:, :n_kv], q_out=q_out, rope=kvd.RopeTable(hd))
        torch.cuda.synchronize()
        assert ok_q() and all(ok() for _, ok in parts)


@pytest.mark.parametrize("dtype,hd,softcap", [("bf16", 128, 0.0), ("f16", 64, 0.0), ("bf16", 64, 20.0), ("f16", 128, 20.0)])
def test_what_nobody_holds_leaves_no_trace(env, dtype, hd, softcap):
    """The same bits whatever lies behind the requests' rows: zeros, the largest code, NaN; and in free pages, their scales too."""
    torch, kvd = env
    lens, new, page = [300, 17, 1000, 5], [1, 17, 300, 4], 64
    outs = []
    for byte, scale in ((0x00, 1.0), (0x7e, 2.0 ** 60), (0x7f, float("nan"))):
        cache, _ = _poisoned8(torch, kvd, lens, 2, hd, page, 5)
        for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            raw = c.view(torch.uint8)
            raw.copy_(torch.where(raw == 0x7f, torch.full_like(raw, byte), raw))
            s.nan_to_num_(scale) if scale == scale else None
        q = (torch.randn(sum(new), 8, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)) * 4).to(_dt(torch, dtype))
        plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
        outs.append(kvd.paged_attention(q, cache, plan, softcap=softcap))
        assert cache.device_error() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and not bool(torch.isnan(outs[0]).any())


def test_a_query_that_is_no_number_is_its_own(env):
    """Infinities and NaN in one row of q: that row's output is NaN, all others as they were."""
    torch, kvd = env
    for lens, new in (([700], [3]), ([700], [200])):
        cache, _ = _poisoned8(torch, kvd, lens, 2, 128, 16, 9)
        for dt in (torch.bfloat16, torch.float16):
            q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)).to(dt)
            plan = kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)
            want = kvd.paged_attention(q, cache, plan)
            for bad in (math.nan, math.inf, -math.inf):
                y = q.clone()
                y[1, 2, 77] = bad
                got = kvd.paged_attention(y, cache, plan)
                assert bool(torch.isnan(got[1, 2]).all())
                got[1, 2] = want[1, 2]
                assert torch.equal(got, want)


def test_pages_may_be_shared_and_queries_broadcast(env):
    """Two requests with one beginning, and one query row for all heads."""
    torch, kvd = env
    cache, rows = _poisoned8(torch, kvd, [128, 200], 2, 64, 64, 15)
    table = cache.block_table.clone()
    table[1, 0] = table[0, 0]
    shared = kvd.PagedKvCache.of(cache.k, cache.v, table, cache.seq_len, k_scale=cache.k_scale, v_scale=cache.v_scale)
    k = torch.cat([rows[0][0][:64], rows[1][0][64:]])
    v = torch.cat([rows[0][1][:64], rows[1][1][64:]])
    row = torch.randn(2, 1, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    q = row.expand(2, 8, 64)
    out = kvd.paged_attention(q, shared, kvd.PagedPlan(_i32(torch, [0, 1, 2]), cache.seq_len))
    v_top = float(cache.v_scale.nan_to_num(0).max())
    _check8(torch, out[:1], _attend8(torch, q[:1], *rows[0], 128, 1 / 8), v_top)
    _check8(torch, out[1:], _attend8(torch, q[1:], k, v, 200, 1 / 8), v_top)
    got = kvd.paged_read(shared, _i32(torch, [0, 0, 200]), 200, dtype=torch.float32)
    assert torch.equal(got[0], k.float()) and torch.equal(got[1], v.float())
