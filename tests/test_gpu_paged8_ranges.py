"""Pages of 8-bit codes on the GPU at the ends of what is allowed.  References and tolerances are those of test_gpu_paged8.py; what a test adds to
them stands beside it.
"""

import math

import numpy as np
import pytest
from test_gpu_paged import _dt, _i32
from test_gpu_paged8 import LOW, _attend8, _check8, _poisoned8, env  # noqa: F401

pytestmark = pytest.mark.gpu


def _plan_of(torch, kvd, cache, new):
    return kvd.PagedPlan(_i32(torch, [0] + np.cumsum(new).tolist()), cache.seq_len)


def _zero_keys(torch, cache, rows, b, page, places):
    """Pages of request b whose keys are all zero, as the writer leaves them: codes 0, the smallest scale."""
    for j in places:
        p, n = int(cache.block_table[b, j]), rows[b][0].shape[0]
        cache.k.view(torch.uint8)[p, :, : max(0, min(page, n - j * page))] = 0
        cache.k_scale[p] = LOW
        rows[b][0][j * page:(j + 1) * page] = 0


@pytest.mark.parametrize("size,scale,softcap", [(2.0 ** -100, None, 0.0), (2.0 ** -100, None, 20.0), (1.0, 1e-30, 0.0), (1.0, None, 1e25), (2.0 ** -60, 1e-20, 3.0)])
@pytest.mark.parametrize("hd,window", [(128, 0), (64, 0), (128, 100)])
def test_small_scores_over_pages_of_zeros(env, size, scale, softcap, hd, window):  # noqa: F811
    """Scores times a page's smallest scale leave f32: what is hidden stays hidden, what is seen weighs the same."""
    torch, kvd = env
    scale = hd ** -0.5 if scale is None else scale
    for lens, new in (([70], [3]), ([300], [200]), ([260], [1])):
        cache, rows = _poisoned8(torch, kvd, lens, 2, hd, 16, 17)
        last = (lens[0] - 1) // 16
        _zero_keys(torch, cache, rows, 0, 16, {last, last - 1, last // 2, 1, 10 % (last + 1)})
        for dt in (torch.bfloat16, torch.float16):
            if size < 2.0 ** -20 and dt is torch.float16:
                continue
            q = (torch.randn(sum(new), 8, hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(18)) * size).to(dt)
            out = kvd.paged_attention(q, cache, _plan_of(torch, kvd, cache, new), scale=scale, window=window, softcap=softcap)
            assert cache.device_error() == 0
            # (a cap of 1e25 is no cap to scores of this size: its tolerance, 2^-20 of it, would say nothing)
            want = _attend8(torch, q, *rows[0], lens[0], scale, window, softcap if softcap < 1e10 else 0.0)
            _check8(torch, out, want, float(cache.v_scale.nan_to_num(0).max()))


PATTERNS = {
    "small first": lambda i, n: -64 if 2 * i < n else 64,
    "large first": lambda i, n: 64 if 2 * i < n else -64,
    "in turn": lambda i, n: 64 if i % 2 else -64,
    "steps": lambda i, n: (-64, 0, 64, 0, -30, 33)[i % 6],
    "one large": lambda i, n: 64 if i == n // 3 else -64,
}


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("pattern", list(PATTERNS))
@pytest.mark.parametrize("hd,lens,new", [(128, 300, 1), (64, 300, 3), (128, 9000, 1), (64, 20011, 2), (128, 700, 200), (64, 9000, 300), (128, 3000, 64)])
def test_scales_of_v_at_both_ends_of_their_range(env, hd, lens, new, pattern, sinks):  # noqa: F811
    """A weight counts in the sum whatever scale its row of V has: scales 2^-64 and 2^64, in tiles, inside tiles and in pieces of one request."""
    torch, kvd = env
    page, pages = 16, -(-lens // 16)
    cache, rows = _poisoned8(torch, kvd, [lens], 2, hd, page, 23)
    for i in range(pages):
        p = int(cache.block_table[0, i])
        to = 2.0 ** PATTERNS[pattern](i, pages)
        rows[0][1][i * page:(i + 1) * page] *= (to / cache.v_scale[p].double())[None, :, None]
        cache.v_scale[p] = to
    g = torch.Generator(device="cuda").manual_seed(24)
    sink = torch.randn(8, generator=g, device="cuda") * 3 + math.log(lens) if sinks else None
    for size, softcap in ((0.0, 0.0), (1.5, 0.0), (4.0, 6.0)):
        q = (torch.randn(new, 8, hd, generator=g, device="cuda") * size).bfloat16()
        out = kvd.paged_attention(q, cache, _plan_of(torch, kvd, cache, [new]), softcap=softcap, sinks=sink)
        assert cache.device_error() == 0
        _check8(torch, out, _attend8(torch, q, *rows[0], lens, hd ** -0.5, 0, softcap, sink), 2.0 ** 64)


@pytest.mark.parametrize("softcap", [1e15, 1e20, 1e25, 1e33, 1e36, 7e36, 3e38])
def test_caps_out_of_reach_change_nothing(env, softcap):  # noqa: F811
    """Scores of some hundreds under caps of any size: right to 2^-19 of themselves, as capped scores are."""
    torch, kvd = env
    for lens, new in (([400], [3]), ([500], [150])):
        for dt in (torch.bfloat16, torch.float16):
            cache, rows = _poisoned8(torch, kvd, lens, 2, 128, 32, 29)
            q = (torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(30)) * 40).to(dt)
            scale = 128 ** -0.5 if softcap < 1e38 else 1.0
            if softcap >= 1e38:
                q = (q.float() * 128 ** -0.5).to(dt)
                softcap = 2.3e38  # log2 e times it is still a number
            out = kvd.paged_attention(q, cache, _plan_of(torch, kvd, cache, new), scale=scale, softcap=softcap)
            assert cache.device_error() == 0
            ref, size, slack = _attend8(torch, q, *rows[0], lens[0], scale)
            top = max(float((q[:, h].double() @ rows[0][0][:, h // 4].T).abs().max()) * scale for h in range(8))
            _check8(torch, out, (ref, size, slack + 2 * 2.0 ** -19 * top), float(cache.v_scale.nan_to_num(0).max()))


def test_caps_below_every_score(env):  # noqa: F811
    """A cap so small that score / cap leaves f32: weights are all alike, keys of zeros among them."""
    torch, kvd = env
    for lens, new in (([400], [3]), ([500], [150])):
        cache, rows = _poisoned8(torch, kvd, lens, 2, 128, 32, 31)
        cache.k_scale *= 2.0 ** 30
        pair = rows[0][0] * 2.0 ** 30, rows[0][1]
        raw = cache.k.view(torch.uint8)
        for i in range(3, lens[0], 7):
            raw[int(cache.block_table[0, i // 32]), :, i % 32] = 0
            pair[0][i] = 0
        for dt in (torch.bfloat16, torch.float16):
            q = torch.randn(sum(new), 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(32)).to(dt)
            out = kvd.paged_attention(q, cache, _plan_of(torch, kvd, cache, new), softcap=1e-36)
            want, size, slack = _attend8(torch, q, *pair, lens[0], 128 ** -0.5, 0, 1e-36)
            # (a score's own error is that of its tanh, of which 1e-36 is left)
            _check8(torch, out, (want, size, torch.full_like(slack, 2.0 ** -20)), float(cache.v_scale.nan_to_num(0).max()))


def test_rows_that_see_nothing_are_zero_whatever_q_is(env):  # noqa: F811
    """New rows that stand before the start of their request, with infinities and NaN in q."""
    torch, kvd = env
    for lens, new in (([3], [5]), ([130], [400]), ([0], [40])):
        for dt, sinks, softcap in ((torch.bfloat16, False, 0.0), (torch.float16, True, 0.0), (torch.bfloat16, True, 20.0)):
            cache, rows = _poisoned8(torch, kvd, lens, 2, 128, 16, 37)
            q = torch.randn(new[0], 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(38)).to(dt)
            hidden = new[0] - lens[0]
            q[0, :, 3] = math.nan
            q[hidden - 1, 2, 77] = math.inf
            sink = torch.randn(8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(39)) if sinks else None
            out = kvd.paged_attention(q, cache, _plan_of(torch, kvd, cache, new), sinks=sink, softcap=softcap)
            assert cache.device_error() == 0 and not out[:hidden].any()
            if lens[0]:
                want = _attend8(torch, q[hidden:], *rows[0], lens[0], 128 ** -0.5, 0, softcap, sink)
                _check8(torch, out[hidden:], want, float(cache.v_scale.nan_to_num(0).max()))


def _rounded(x, bits):
    """f64 rounded to so many significant bits, to nearest even."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


@pytest.mark.parametrize("to,bits", [("bf16", 8), ("f16", 11), ("f32", 24)])
def test_odd_scales_are_read_with_one_rounding(env, to, bits):  # noqa: F811
    """code * scale just beside the middle of two numbers of the type, where f32 already rounds to the middle: a second rounding would go to the even one."""
    torch, kvd = env
    scales, b = [], min(bits, 11)
    for c in (9, 11, 13, 15):  # significands of codes
        for k in range(1 << (b - 1), 1 << b, 1 if b == 8 else 11):
            middle = (2 * k + 1) << (27 - b)  # 28 bits, of which f32 keeps 24
            m = round(middle / c)
            off = c * m - middle
            if (1 << 23) <= m < (1 << 24) and off != 0 and (off > 0) == (k % 2 == 0):
                scales.append(m * 2.0 ** -24)
    assert len(scales) >= 20
    scales = np.array(scales[:200])
    n = len(scales)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(4, 64).repeat(n, 4, 1).view(n, 1, 16, 64)
    codes[(codes & 127) == 127] = 0
    one = torch.from_numpy(scales).float().cuda().view(n, 1)
    cache = kvd.PagedKvCache.of(codes.view(torch.float8_e4m3fn), codes.clone().view(torch.float8_e4m3fn), torch.arange(n, dtype=torch.int32, device="cuda").view(1, n),
                                _i32(torch, [16 * n]), k_scale=one, v_scale=one.clone())
    got = kvd.paged_read(cache, _i32(torch, [0, 16 * n]), 16 * n, dtype=_dt(torch, to))
    values = codes.view(torch.float8_e4m3fn).double().cpu().numpy().reshape(n, 16, 64)
    exact = values * scales[:, None, None]
    twice = _rounded(exact.astype(np.float32).astype(np.float64), bits)
    want = _rounded(exact, bits)
    assert to == "f32" or (twice != want).sum() >= n // 2  # what is tested happens
    for x in got:
        assert np.array_equal(x.double().cpu().numpy().reshape(n, 16, 64), want)


@pytest.mark.parametrize("total,new,group,dtype", [(200000, 1, 4, "bf16"), (200000, 1, 8, "f16"), (200000, 1, 16, "f16"), (200000, 3, 4, "bf16"), (30000, 600, 4, "bf16"),
                                                   (30000, 600, 2, "f16")])
def test_launches_given_up_within_a_run_of_tiles(env, total, new, group, dtype):  # noqa: F811
    """Blocks with tens of tiles, given up long after their first and long before their last: the launch ends and says so, and the next call is right."""
    torch, kvd = env
    from kv_cache_decode_attention_gb300 import _abi

    n_kv, hd, page = 8, 128, 128
    pages = -(-total // page)
    cache = kvd.PagedKvCache(pages, page, n_kv, hd, 1, pages, dtype=torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(43)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).copy_(torch.randint(0, 0x7f, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    cache.k_scale.fill_(2.0 ** -10)
    cache.block_table.copy_(torch.randperm(pages, generator=g, device="cuda").int()[None])
    cache.seq_len.fill_(total)
    q = torch.randn(new, n_kv * group, hd, generator=g, device="cuda").to(_dt(torch, dtype))
    plan = _plan_of(torch, kvd, cache, [new])
    want = kvd.paged_attention(q, cache, plan)
    assert cache.device_error() == 0
    graph, times = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for _ in range(8):
            kvd.paged_attention(q, cache, plan)
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / 8 * 1e6)
    whole = sorted(times)[2]  # ns of a call's launches: a block is at its tiles for most of it
    try:
        for cta in (0, 37, 95, 151):
            for share in (0.15, 0.25, 0.35):
                assert _abi.lib().kvd_test_give_up(cta, int(share * whole)) == 0
                kvd.paged_attention(q, cache, plan)
                _abi.lib().kvd_test_give_up(-1, 0)
                assert cache.device_error() == 1, (cta, share)
                assert torch.equal(kvd.paged_attention(q, cache, plan), want) and cache.device_error() == 0
            for share in (0.7, 0.8, 0.9, 1.0, 1.5):  # about its end
                assert _abi.lib().kvd_test_give_up(cta, int(share * whole)) == 0
                out = kvd.paged_attention(q, cache, plan)
                _abi.lib().kvd_test_give_up(-1, 0)
                assert cache.device_error() == 1 or torch.equal(out, want)
            assert _abi.lib().kvd_test_give_up(cta, 10 ** 9) == 0
            assert torch.equal(kvd.paged_attention(q, cache, plan), want) and cache.device_error() == 0
    finally:
        _abi.lib().kvd_test_give_up(-1, 0)


@pytest.mark.parametrize("value,low", [(1.0, -8), (2.0 ** 15, 9)])
@pytest.mark.parametrize("dtype,hd,group", [("bf16", 128, 4), ("f16", 64, 16), ("f16", 128, 5), ("bf16", 64, 1)])
def test_one_number_everywhere_comes_out_as_itself(env, value, low, dtype, hd, group):  # noqa: F811
    """V is one number, held at scales 2^low .. 2^(low + 5), and zero in some pages: what comes out is the number times the weight of the others.
    A weight times its scale is held to 2^-22 of the largest of its 128 rows, so at scales 2^5 apart the output is off by 128 * 2^-22 * 2^5 of
    the number at most for that."""
    torch, kvd = env
    lens, new, page = [900, 5000, 3, 700, 2000], [1, 2, 3, 300, 33], 32
    r = np.random.default_rng(hd + group)
    for window, softcap, sinks, size in ((0, 0.0, False, 1.5), (600, 0.0, True, 1.5), (0, 20.0, True, 4.0), (0, 0.0, False, 0.0)):
        cache, rows = _poisoned8(torch, kvd, lens, 2, hd, page, 47)
        raw, shares = cache.v.view(torch.uint8), []
        for b, n in enumerate(lens):
            v = torch.full((n,), value, dtype=torch.float64, device="cuda")
            for j in range(-(-n // page)):
                p, held = int(cache.block_table[b, j]), min(page, n - j * page)
                e = int(r.integers(low, low + 6))
                zero = r.random() < 0.15
                cache.v_scale[p] = LOW if zero else 2.0 ** e
                raw[p, :, :held] = 0 if zero else int(torch.tensor(value * 2.0 ** -e).to(torch.float8_e4m3fn).view(torch.uint8))
                if zero:
                    v[j * page:j * page + held] = 0
            shares.append(v)
        g = torch.Generator(device="cuda").manual_seed(48)
        q = (torch.randn(sum(new), 2 * group, hd, generator=g, device="cuda") * size).to(_dt(torch, dtype))
        sink = torch.randn(2 * group, generator=g, device="cuda") if sinks else None
        out = kvd.paged_attention(q, cache, _plan_of(torch, kvd, cache, new), window=window, softcap=softcap, sinks=sink)
        assert cache.device_error() == 0
        at, half = 0, float(torch.finfo(out.dtype).eps) / 2
        for b, n in enumerate(new):
            v = shares[b][:, None, None].expand(lens[b], 2, hd)
            want, size_of, slack = _attend8(torch, q[at:at + n], rows[b][0], v, lens[b], hd ** -0.5, window, softcap, sink)
            tol = (half + slack * (1 + half)) * size_of * (1 + half) + half * want.abs() + value * 2.0 ** -10
            assert bool(((out[at:at + n].double() - want).abs() <= tol).all())
            at += n
