"""Paged serving, the part that needs no GPU: frequency tables against their
formulas and every refusal of the entry points (validation comes before any
launch, so the pointers below are never dereferenced)."""

import ctypes as C
import math
import struct

import pytest

FAKE = 1 << 20


@pytest.fixture(scope="module")
def abi():
    from kv_cache_decode_attention_gb300 import _abi
    from kv_cache_decode_attention_gb300.build import build

    build()
    return _abi


GOOD = dict(rot_dim=128, layout=1, scaling=0, pad=0, base=10000.0, factor=1.0, original_len=4096.0, beta_fast=32.0, beta_slow=1.0,
            low_freq_factor=1.0, high_freq_factor=4.0, attention_factor=0.0)


def _init(abi, **kw):
    cfg = abi.kvd_rope_config(**{**GOOD, **kw})
    R = abi.kvd_rope()
    return abi.lib().kvd_rope_init(C.byref(R), C.byref(cfg)), R


def _fields(R):
    """factor and the 64-bit turns of an initialised table."""
    raw = bytes(R)
    return struct.unpack_from("f", raw, 12)[0], struct.unpack_from("256Q", raw, 16)


def _wanted(c):
    rot, base, factor = c["rot_dim"], c["base"], c["factor"]
    if c["scaling"] == 2:
        base *= factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if c["scaling"] == 1:
            f /= factor
        elif c["scaling"] == 3:
            dim = lambda turns: rot * math.log(c["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            low, high = max(math.floor(dim(c["beta_fast"])), 0), min(math.ceil(dim(c["beta_slow"])), rot - 1)
            r = min(max((i - low) / max(high - low, 1e-3), 0), 1)
            f = f / factor * r + f * (1 - r)
        elif c["scaling"] == 4:
            w = c["original_len"] * f / (2 * math.pi)
            m = min(max((w - c["low_freq_factor"]) / (c["high_freq_factor"] - c["low_freq_factor"]), 0), 1)
            f = f / factor * (1 - m) + f * m
        out.append(f)
    return out


@pytest.mark.parametrize("kw", [dict(), dict(rot_dim=2), dict(rot_dim=512, layout=0), dict(scaling=1, factor=4.0), dict(scaling=2, factor=8.0),
                                dict(scaling=3, factor=8.0), dict(scaling=3, factor=1.0, rot_dim=6), dict(scaling=4, factor=8.0, original_len=8192.0),
                                dict(scaling=4, factor=8.0, base=500000.0)])
def test_rope_table_matches_its_formula(abi, kw):
    st, R = _init(abi, **kw)
    assert st == abi.OK
    c = {**GOOD, **kw}
    mul, turns = _fields(R)
    want_mul = 0.1 * math.log(c["factor"]) + 1 if c["scaling"] == 3 else 1.0
    assert abs(mul - want_mul) <= 2 ** -24 * want_mul
    for f, t in zip(_wanted(c), turns):
        # two evaluations of pow, log and a few products in f64: some 2^-53 of
        # relative error each, 64 of them at most
        assert abs(t / 2 ** 64 * 2 * math.pi - f) <= 64 * 2 ** -53 * f + 2 ** -60
    assert _init(abi, attention_factor=0.5)[0] == abi.OK and _fields(_init(abi, attention_factor=0.5)[1])[0] == 0.5


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=514), dict(rot_dim=-2), dict(layout=2), dict(scaling=5), dict(scaling=-1),
                                dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(scaling=1, factor=0.5),
                                dict(scaling=1, factor=float("inf")), dict(scaling=2, factor=2.0, rot_dim=2), dict(scaling=3, factor=2.0, original_len=0.0),
                                dict(scaling=3, factor=2.0, beta_fast=1.0), dict(scaling=3, factor=2.0, beta_slow=0.0), dict(scaling=4, factor=2.0, high_freq_factor=1.0),
                                dict(scaling=4, factor=2.0, low_freq_factor=-1.0), dict(attention_factor=-1.0), dict(attention_factor=float("nan"))])
def test_rope_table_refusals(abi, kw):
    assert _init(abi, **kw)[0] == abi.EINVAL
    assert abi.lib().kvd_rope_init(None, None) == abi.EINVAL


def _rows(abi, data=FAKE, tok=1024, head=128):
    return C.byref(abi.kvd_rows(data, tok, head))


def test_rope_apply_refusals(abi):
    L = abi.lib()
    R = _init(abi)[1]

    def call(R=C.byref(R), q=0, qo=0, n_q=8, k=0, ko=0, n_kv=8, hd=128, dtype=2, pos=FAKE, n=4):
        q, qo, k, ko = (_rows(abi) if x == 0 else x for x in (q, qo, k, ko))
        return L.kvd_rope_apply(R, q, qo, n_q, k, ko, n_kv, hd, dtype, pos, n, None)

    assert call(n=0) == abi.OK  # nothing to do, nothing launched
    for bad in (dict(R=None), dict(R=C.byref(abi.kvd_rope())), dict(q=None), dict(qo=None), dict(q=None, qo=None, k=None, ko=None), dict(n_q=0),
                dict(n_kv=1025), dict(hd=64), dict(hd=520), dict(dtype=3), dict(pos=None), dict(n=-1), dict(n=1 << 31), dict(q=_rows(abi, 0)),
                dict(q=_rows(abi, FAKE + 1)), dict(qo=_rows(abi, tok=2048)), dict(q=_rows(abi, tok=-1024)), dict(k=_rows(abi, head=-1)),
                dict(qo=_rows(abi, 2 * FAKE, tok=0)), dict(ko=_rows(abi, 2 * FAKE, head=0))):
        assert call(**bad) == abi.EINVAL, bad


def test_plan_refusals(abi):
    L = abi.lib()
    names = ["seq_len", "keep_len", "new_len", "n_seq", "n_pages", "page_size", "table", "max_pages", "free", "n_free", "len_out", "free_out", "cu",
             "positions", "slots", "n_tokens", "err"]
    good = dict(zip(names, [FAKE, None, FAKE, 4, 64, 16, FAKE, 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 32, FAKE]))

    def call(**kw):
        return L.kv_paged_plan(*{**good, **kw}.values(), None)

    for bad in (dict(seq_len=None), dict(new_len=None), dict(table=None), dict(free=None), dict(n_free=None), dict(len_out=None), dict(free_out=None),
                dict(cu=None), dict(positions=None), dict(slots=None), dict(err=None), dict(n_seq=0), dict(n_seq=8193), dict(n_pages=0),
                dict(n_pages=1 << 27), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(max_pages=0), dict(max_pages=1 << 27),
                dict(max_pages=(1 << 27) - 63), dict(n_tokens=-1), dict(n_tokens=1 << 31)):
        assert call(**bad) == abi.EINVAL, bad


def test_append_refusals(abi):
    L = abi.lib()
    R = _init(abi)[1]
    wide = _init(abi, rot_dim=256)[1]

    def call(R=C.byref(R), q=0, qo=0, n_q=8, k=0, v=0, n_kv=8, hd=128, it=2, pt=2, pos=FAKE, slots=FAKE, n=4, kp=FAKE, vp=FAKE, n_pages=64, page=16,
             err=FAKE):
        q, qo, k, v = (_rows(abi) if x == 0 else x for x in (q, qo, k, v))
        return L.kv_paged_append(R, q, qo, n_q, k, v, n_kv, hd, it, pt, pos, slots, n, kp, vp, n_pages, page, err, None)

    assert call(n=0) == abi.OK and call(n=0, R=None) == abi.OK and call(n=0, q=None, qo=None) == abi.OK and call(n=0, it=0, qo=_rows(abi, 2 * FAKE)) == abi.OK
    for bad in (dict(R=C.byref(abi.kvd_rope())), dict(R=C.byref(wide)), dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(n_q=0), dict(n_kv=0),
                dict(hd=96), dict(hd=256), dict(it=1), dict(it=3), dict(pt=0), dict(pos=None), dict(slots=None), dict(n=-1), dict(kp=None), dict(vp=FAKE + 8),
                dict(n_pages=0), dict(n_pages=1 << 27), dict(page=24), dict(page=256), dict(err=None), dict(it=0), dict(qo=_rows(abi, tok=2048))):
        assert call(**bad) == abi.EINVAL, bad


def test_attention_refusals(abi):
    L = abi.lib()
    n = C.c_int64(0)
    ws = lambda t, n_q=32, n_kv=8, hd=128: L.paged_attention_workspace_bytes(t, n_q, n_kv, hd, C.byref(n))  # noqa: E731
    assert ws(4096) == abi.OK
    need = n.value
    assert ws(1) == abi.OK and 0 < n.value < need
    for bad in ((-1,), (1, 31), (1, 8, 0), (1, 8, 8, 96), (1, 136, 8), (1, 4, 8)):
        assert ws(*bad) == abi.EINVAL, bad
    assert L.paged_attention_workspace_bytes(1, 8, 8, 128, None) == abi.EINVAL

    def call(q=0, out=0, n=64, n_q=8, n_kv=8, hd=128, dt=2, kp=FAKE, vp=FAKE, n_pages=64, page=16, table=FAKE, width=8, cu=FAKE, lens=FAKE, n_seq=4,
             scale=0.1, window=0, softcap=0.0, sinks=None, w=FAKE, wb=1 << 40, err=FAKE):
        q, out = _rows(abi) if q == 0 else q, _rows(abi, 2 * FAKE) if out == 0 else out
        return L.paged_attention(q, out, n, n_q, n_kv, hd, dt, kp, vp, n_pages, page, table, width, cu, lens, n_seq, scale, window, softcap, sinks, w, wb, err, None)

    assert call(n=0) == abi.OK
    assert call(n=0, q=_rows(abi, 0, tok=3, head=128)) == abi.OK  # the stride of an axis with one entry is not looked at
    inf, nan = float("inf"), float("nan")
    for bad in (dict(q=None), dict(out=None), dict(out=_rows(abi)), dict(q=_rows(abi, FAKE + 8)), dict(q=_rows(abi, tok=1028)), dict(out=_rows(abi, 2 * FAKE, head=132)),
                dict(q=_rows(abi, tok=-1024)), dict(n=-1), dict(n_q=12), dict(n_q=136), dict(n_kv=0), dict(hd=32), dict(dt=0), dict(dt=7), dict(kp=None), dict(vp=FAKE + 8),
                dict(n_pages=0), dict(n_pages=1 << 24), dict(page=12), dict(page=256), dict(table=None), dict(width=0), dict(width=1 << 27),
                dict(width=(1 << 27) - 63), dict(out=_rows(abi, 2 * FAKE, tok=0)), dict(out=_rows(abi, 2 * FAKE, head=0)), dict(scale=3e38), dict(softcap=3e38),
                dict(softcap=1e-38, scale=10.0), dict(cu=None), dict(lens=None), dict(n_seq=0), dict(scale=0.0), dict(scale=-0.1), dict(scale=nan), dict(scale=inf), dict(window=-1), dict(softcap=-1.0), dict(softcap=nan), dict(sinks=FAKE + 2),
                dict(w=None), dict(w=FAKE + 16), dict(wb=1024), dict(err=None)):
        assert call(**bad) == abi.EINVAL, bad
    assert L.kv_paged_device_error(None, 0, None) == abi.EINVAL


def test_calls_without_rows_do_nothing(abi):
    """No rows: no pointer is needed, nothing is launched."""
    L = abi.lib()
    R = _init(abi)[1]
    null = lambda: C.byref(abi.kvd_rows(None, 0, 0))  # noqa: E731
    assert L.kvd_rope_apply(C.byref(R), null(), null(), 8, None, None, 0, 128, 2, None, 0, None) == abi.OK
    assert L.kv_paged_append(C.byref(R), null(), null(), 8, null(), null(), 8, 128, 0, 2, None, None, 0, FAKE, FAKE, 64, 16, FAKE, None) == abi.OK
    assert L.paged_attention(null(), null(), 0, 8, 8, 128, 2, FAKE, FAKE, 64, 16, FAKE, 8, FAKE, FAKE, 4, 0.1, 0, 0.0, None, None, 0, FAKE, None) == abi.OK


def test_give_up_refusals(abi):
    L = abi.lib()
    assert L.kvd_test_give_up(-1, 0) == abi.OK
    for bad in ((152, 0), (0, -1), (0, 10 ** 9 + 1)):
        assert L.kvd_test_give_up(*bad) == abi.EINVAL, bad


VIEWS = r"""
#include "kvd_views.h"
using namespace kvd;
static View view(const long long *v) { return {uintptr_t(v[0]), v[1], v[2], v[3], v[4], v[5]}; }
extern "C" int apart(const long long *a, const long long *b) { return views_apart(view(a), view(b)); }
extern "C" int rows(const long long *a) { return rows_apart(view(a)); }
"""


@pytest.fixture(scope="module")
def views(tmp_path_factory):
    """kvd_views.h as a library of its own."""
    import subprocess

    from kv_cache_decode_attention_gb300.build import CSRC

    d = tmp_path_factory.mktemp("views")
    (d / "v.cpp").write_text(VIEWS)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "v.cpp"), "-o", str(d / "v.so")], check=True)
    lib = C.CDLL(str(d / "v.so"))
    arr = lambda v: (C.c_longlong * 6)(*v)  # noqa: E731
    return (lambda a, b: bool(lib.apart(arr(a), arr(b)))), (lambda a: bool(lib.rows(arr(a))))


def _bytes(v):
    at, t, h, nt, nh, row = v
    return [at + i * t + j * h + c for i in range(nt) for j in range(nh) for c in range(row)]


def test_views_that_share_bytes_are_never_taken_for_apart(views):
    """Drawn views of any strides, byte by byte."""
    import random

    apart, rows = views
    rng = random.Random(4)

    def draw():
        nt, nh, row = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 5)
        return [rng.randint(64, 110), rng.randint(0, 24) if nt > 1 else 0, rng.randint(0, 24) if nh > 1 else 0, nt, nh, row]

    said = 0
    for _ in range(30000):
        a, b = draw(), draw()
        shared = bool(set(_bytes(a)) & set(_bytes(b)))
        assert not (shared and apart(a, b)), (a, b)
        assert apart(a, b) == apart(b, a)
        once = len(set(_bytes(a))) == len(_bytes(a))
        assert not (rows(a) and not once), a
        said += apart(a, b)
    assert said > 5000


def test_slices_of_one_array_are_known(views):
    """Heads, channels, tokens and transpositions of one array: told apart exactly."""
    import random

    apart, rows = views
    rng = random.Random(5)
    seen = set()
    for _ in range(6000):
        T, H, D = rng.randint(1, 5), rng.randint(1, 6), rng.randint(1, 6)
        flip = rng.random() < 0.3  # heads outermost

        def part():
            t0, h0, d0 = rng.randrange(T), rng.randrange(H), rng.randrange(D)
            nt, nh, nd = rng.randint(1, T - t0), rng.randint(1, H - h0), rng.randint(1, D - d0)
            ts, hs = (D, T * D) if flip else (H * D, D)
            return [1000 + t0 * ts + h0 * hs + d0, ts if nt > 1 else 0, hs if nh > 1 else 0, nt, nh, nd], (t0, t0 + nt, h0, h0 + nh, d0, d0 + nd)

        (a, x), (b, y) = part(), part()
        shared = bool(set(_bytes(a)) & set(_bytes(b)))
        assert rows(a) and rows(b)
        # boxes that differ in two axes or more are apart by any of them; the ranges or one modulus shows it unless an axis of one
        # entry hides the array's stride
        if shared:
            assert not apart(a, b)
        elif min(a[3], b[3]) > 1 and min(a[4], b[4]) > 1:
            assert apart(a, b), (a, b, x, y)
        seen.add((shared, apart(a, b)))
    assert {(True, False), (False, True)} <= seen


def test_attention_outputs_that_share_memory_are_refused(abi):
    """Refused before anything is launched: out on q, on the pages, or on itself."""
    L = abi.lib()
    far = 1 << 32

    def call(q, out, n=64, kp=far, vp=2 * far):
        return L.paged_attention(q, out, n, 8, 8, 128, 2, kp, vp, 64, 16, FAKE, 8, FAKE, FAKE, 4, 0.1, 0, 0.0, None, FAKE, 1 << 40, FAKE, None)

    rows = lambda at, tok=1024, head=128: _rows(abi, at, tok, head)  # noqa: E731
    q = rows(FAKE, 4096)
    for out in (rows(FAKE, 4096), rows(FAKE + 256, 4096), rows(FAKE + 7 * 256, 4096), rows(FAKE - 256, 4096), rows(FAKE + 8192, 4096), rows(FAKE + 128, 4096),
                rows(FAKE, 2048), rows(far), rows(far + (64 * 16 * 8 * 256) - 16), rows(2 * far + 4096), rows(8 * FAKE, 1024, 64), rows(8 * FAKE, 64, 1024),
                rows(8 * FAKE, 512), rows(8 * FAKE, 960)):
        assert call(q, out) == abi.EINVAL


def test_rotated_outputs_that_share_memory_are_refused(abi):
    """Without a GPU a call that is taken fails at its launch (ECUDA), so a refusal is one of the arguments."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    L = abi.lib()
    R = C.byref(_init(abi)[1])
    M = 1 << 24
    r = lambda at, tok=1024, head=128: _rows(abi, at, tok, head)  # noqa: E731

    def rope(q, qo, k=None, ko=None, dtype=2):
        return L.kvd_rope_apply(R, q, qo, 8, k, ko, 8, 128, dtype, FAKE, 64, None)

    def append(q, qo, k=None, v=None, kp=64 * M, vp=128 * M, it=2):
        k, v = r(4 * M) if k is None else k, r(8 * M) if v is None else v
        return L.kv_paged_append(R, q, qo, 8, k, v, 8, 128, it, 2, FAKE, FAKE, 64, kp, vp, 64, 16, FAKE, None)

    W = 4096  # heads of 128 of one projection: q 0 .. 7, k 8 .. 15, v 16 .. 23
    q, k, v = (r(M + i * 8 * 256, W) for i in range(3))
    for call in (lambda: rope(r(M), r(M)), lambda: rope(r(M), r(2 * M)), lambda: rope(q, q, k, k), lambda: rope(q, v, k, r(2 * M)),
                 lambda: rope(r(M, 128, 8192), r(M, 128, 8192)), lambda: rope(r(M, 0, 0), r(2 * M)), lambda: append(q, q, k, v), lambda: append(r(M), r(2 * M)),
                 lambda: append(r(M), r(2 * M), q, q), lambda: append(None, None, k, k)):
        assert call() == abi.ECUDA
    for call in (lambda: rope(r(M), r(M + 256)), lambda: rope(r(M), r(M - 256)), lambda: rope(r(M), r(M + 2048)), lambda: rope(r(M), r(M, 2048)),
                 lambda: rope(q, k, k, q), lambda: rope(q, q, q, q), lambda: rope(q, r(2 * M), k, r(2 * M)), lambda: rope(q, k, k, r(2 * M)),
                 lambda: rope(r(M), r(2 * M, 1024, 64)), lambda: rope(r(M), r(2 * M, 512)), lambda: rope(r(M), r(2 * M, 64, 128)),
                 lambda: append(q, k, k, v), lambda: append(q, v, k, v), lambda: append(r(M), r(M), it=0), lambda: append(r(M), r(M + 256)),
                 lambda: append(r(64 * M), r(M)), lambda: append(r(M), r(128 * M + 4096)), lambda: append(None, None, r(64 * M + 65536)),
                 lambda: append(None, None, None, r(128 * M)), lambda: append(None, None, kp=64 * M, vp=64 * M), lambda: append(None, None, kp=64 * M, vp=64 * M + 4096)):
        assert call() == abi.EINVAL


def test_attention_refuses_more_requests_than_it_can_walk(abi):
    L = abi.lib()
    call = lambda n_seq, n: L.paged_attention(_rows(abi), _rows(abi, 2 * FAKE), n, 8, 8, 128, 2, FAKE * 64, FAKE * 64, 64, 16, FAKE, 8, FAKE, FAKE, n_seq, 0.1,  # noqa: E731
                                              0, 0.0, None, FAKE, 1 << 40, FAKE, None)
    assert call(1 << 20, 0) == abi.OK  # nothing to do
    for n_seq in ((1 << 20) + 1, 2 ** 31 - 1):
        assert call(n_seq, 0) == abi.EINVAL and call(n_seq, 4) == abi.EINVAL


def _turns_of(c, digits=60):
    """f_i / 2 pi of a config by its formula, with so many digits."""
    from decimal import Decimal as D, localcontext

    with localcontext() as ctx:
        ctx.prec = digits
        two_pi = 2 * D("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
        rot, factor, length = c["rot_dim"], D(c["factor"]), D(c["original_len"])
        log_base = D(c["base"]).ln()
        if c["scaling"] == 2:
            log_base += factor.ln() * rot / (rot - 2)
        if c["scaling"] == 3:
            pair = lambda turns: rot * (length / (D(turns) * two_pi)).ln() / (2 * log_base)  # noqa: E731
            low = max(int(pair(c["beta_fast"]).to_integral_value("ROUND_FLOOR")), 0)
            high = min(int(pair(c["beta_slow"]).to_integral_value("ROUND_CEILING")), rot - 1)
        out = []
        for i in range(rot // 2):
            f = (log_base * (-2 * i) / rot).exp()
            if c["scaling"] == 1:
                f /= factor
            elif c["scaling"] == 3:
                r = min(max((i - low) / max(D(high - low), D("0.001")), D(0)), D(1))
                f = f / factor * r + f * (1 - r)
            elif c["scaling"] == 4:
                lo, hi = D(c["low_freq_factor"]), D(c["high_freq_factor"])
                m = min(max((length * f / two_pi - lo) / (hi - lo), D(0)), D(1))
                f = f / factor * (1 - m) + f * m
            out.append(f / two_pi)
        return out


@pytest.mark.parametrize("scaling", range(5))
def test_rope_table_is_right_to_2_to_the_minus_54_turns(abi, scaling):
    """Against 60 digits.  f <= 1, so f / 2 pi < 0.16: pow, the scaling's products and sums and the division by 2 pi are a few roundings of
    2^-53 of that each."""
    for rot in (4, 64, 70, 128, 512):
        for base in (100.0, 10000.0, 500000.0, 1e7):
            for factor, length in ((1.0, 8192.0), (3.7, 2048.0), (8.0, 4096.0), (32.0, 32768.0)):
                kw = dict(rot_dim=rot, scaling=scaling, base=base, factor=factor, original_len=length)
                st, R = _init(abi, **kw)
                assert st == abi.OK
                for got, want in zip(_fields(R)[1], _turns_of({**GOOD, **kw})):
                    assert abs(got - want * 2 ** 64) <= 2 ** 10, kw
