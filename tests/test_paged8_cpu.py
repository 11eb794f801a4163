"""Pages of 8-bit codes, the part that needs no GPU: every refusal of the entry points (validation comes before any launch, so the
pointers below are never dereferenced)."""

import ctypes as C

import pytest
from test_paged_cpu import FAKE, _init, _rows


@pytest.fixture(scope="module")
def abi():
    from kv_cache_decode_attention_gb300 import _abi
    from kv_cache_decode_attention_gb300.build import build

    build()
    return _abi


def _far(i):
    """Memory that shares nothing with the other pointers of a call."""
    return FAKE + (i << 32)


def test_append_refusals(abi):
    L = abi.lib()
    R, wide = _init(abi)[1], _init(abi, rot_dim=256)[1]

    def call(R=C.byref(R), q=0, qo=0, n_q=8, k=0, v=0, n_kv=8, hd=128, it=2, qt=2, pos=FAKE, slots=FAKE, n=4, kp=_far(1), vp=_far(2), ks=_far(3), vs=_far(4),
             n_pages=64, page=16, err=FAKE):
        q, qo, k, v = (_rows(abi, _far(5 + i)) if x == 0 else x for i, x in enumerate((q, qo, k, v)))
        return L.kv_paged_append_q8(R, q, qo, n_q, k, v, n_kv, hd, it, qt, pos, slots, n, kp, vp, ks, vs, n_pages, page, err, None)

    assert call(n=0) == abi.OK and call(n=0, R=None) == abi.OK and call(n=0, q=None, qo=None, qt=-1) == abi.OK and call(n=0, it=0, qt=1) == abi.OK
    for bad in (dict(R=C.byref(abi.kvd_rope())), dict(R=C.byref(wide)), dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(n_q=0), dict(n_q=1025),
                dict(n_kv=0), dict(n_kv=1025), dict(hd=96), dict(hd=256), dict(it=1), dict(it=3), dict(it=-1), dict(qt=0), dict(qt=3), dict(qt=1), dict(pos=None),
                dict(slots=None), dict(n=-1), dict(n=1 << 31), dict(kp=None), dict(vp=_far(2) + 8), dict(ks=None), dict(vs=None), dict(ks=_far(3) + 2), dict(n_pages=0),
                dict(n_pages=1 << 27), dict(page=24), dict(page=8), dict(page=256), dict(err=None), dict(k=_rows(abi, _far(7) + 1)), dict(v=_rows(abi, _far(8), tok=-8)),
                # what is written shares memory with nothing else
                dict(vp=_far(1)), dict(vs=_far(3)), dict(ks=_far(1)), dict(vp=_far(1) + 64 * 16 * 8 * 128 - 16), dict(k=_rows(abi, _far(1))), dict(v=_rows(abi, _far(4))),
                dict(qo=_rows(abi, _far(2))), dict(q=_rows(abi, _far(2))), dict(qo=_rows(abi, _far(7))), dict(qo=_rows(abi, _far(6), tok=0)),
                dict(q=_rows(abi, _far(6), tok=2048))):
        assert call(**bad) == abi.EINVAL, bad


def test_read_refusals(abi):
    L = abi.lib()

    def call(kp=_far(1), vp=_far(2), ks=_far(3), vs=_far(4), pt=3, n_pages=64, page=16, n_kv=8, hd=128, table=FAKE, width=8, lens=FAKE, start=None, cu=FAKE,
             n_seq=4, ko=0, vo=0, ot=2, n=4, err=FAKE):
        ko, vo = (_rows(abi, _far(5 + i)) if x == 0 else x for i, x in enumerate((ko, vo)))
        return L.kv_paged_read(kp, vp, ks, vs, pt, n_pages, page, n_kv, hd, table, width, lens, start, cu, n_seq, ko, vo, ot, n, err, None)

    assert call(n=0) == abi.OK and call(n=0, pt=2, ks=None, vs=None) == abi.OK and call(n=0, start=FAKE, ot=0) == abi.OK
    for bad in (dict(kp=None), dict(vp=_far(2) + 4), dict(ks=None), dict(vs=None), dict(vs=_far(4) + 1), dict(pt=2), dict(pt=0, ks=None, vs=None), dict(pt=4), dict(ot=3),
                dict(ot=-1), dict(n_pages=0), dict(n_pages=1 << 27), dict(page=20), dict(page=256), dict(n_kv=0), dict(n_kv=1025), dict(hd=96), dict(table=None), dict(width=0),
                dict(lens=None), dict(cu=None), dict(n_seq=0), dict(n_seq=(1 << 20) + 1), dict(ko=None), dict(vo=None), dict(n=-1), dict(n=1 << 31), dict(err=None),
                dict(ko=_rows(abi, _far(5) + 2)), dict(ko=_rows(abi, _far(5), tok=1028)), dict(vo=_rows(abi, _far(6), head=132)), dict(ko=_rows(abi, _far(6))),
                dict(ko=_rows(abi, _far(1))), dict(vo=_rows(abi, _far(3))), dict(ko=_rows(abi, _far(5), tok=0)), dict(vo=_rows(abi, _far(6), head=0))):
        assert call(**bad) == abi.EINVAL, bad


def test_attention_refusals(abi):
    L = abi.lib()
    n = C.c_int64(0)
    ws = lambda t, n_q=32, n_kv=8, hd=128: L.paged_attention_q8_workspace_bytes(t, n_q, n_kv, hd, C.byref(n))  # noqa: E731
    assert ws(4096) == abi.OK
    need = n.value
    assert ws(1) == abi.OK and 0 < n.value < need
    for bad in ((-1,), (1, 31), (1, 8, 0), (1, 8, 8, 96), (1, 136, 8), (1, 4, 8)):
        assert ws(*bad) == abi.EINVAL, bad
    assert L.paged_attention_q8_workspace_bytes(1, 8, 8, 128, None) == abi.EINVAL

    def call(q=0, out=0, n=64, n_q=8, n_kv=8, hd=128, dt=2, kp=_far(1), vp=_far(2), ks=_far(3), vs=_far(4), n_pages=64, page=16, table=FAKE, width=8, cu=FAKE, lens=FAKE,
             n_seq=4, scale=0.1, window=0, softcap=0.0, sinks=None, w=FAKE, wb=1 << 40, err=FAKE):
        q, out = _rows(abi, _far(5)) if q == 0 else q, _rows(abi, _far(6)) if out == 0 else out
        return L.paged_attention_q8(q, out, n, n_q, n_kv, hd, dt, kp, vp, ks, vs, n_pages, page, table, width, cu, lens, n_seq, scale, window, softcap, sinks, w, wb, err, None)

    assert call(n=0) == abi.OK
    inf, nan = float("inf"), float("nan")
    for bad in (dict(q=None), dict(out=None), dict(out=_rows(abi, _far(5))), dict(q=_rows(abi, _far(5) + 8)), dict(q=_rows(abi, _far(5), tok=1028)),
                dict(out=_rows(abi, _far(6), head=132)), dict(q=_rows(abi, _far(5), tok=-1024)), dict(n=-1), dict(n_q=12), dict(n_q=136), dict(n_kv=0), dict(hd=32),
                dict(dt=0), dict(dt=3), dict(kp=None), dict(vp=_far(2) + 8), dict(ks=None), dict(vs=_far(4) + 2), dict(n_pages=0), dict(n_pages=1 << 24), dict(page=12),
                dict(page=256), dict(table=None), dict(width=0), dict(width=1 << 27), dict(out=_rows(abi, _far(6), tok=0)), dict(scale=3e38), dict(softcap=3e38),
                dict(softcap=1e-38, scale=10.0), dict(cu=None), dict(lens=None), dict(n_seq=0), dict(n_seq=(1 << 20) + 1), dict(scale=0.0), dict(scale=nan), dict(scale=inf),
                dict(window=-1), dict(softcap=-1.0), dict(softcap=nan), dict(sinks=FAKE + 2), dict(w=None), dict(w=FAKE + 16), dict(wb=1024), dict(err=None),
                dict(out=_rows(abi, _far(1))), dict(out=_rows(abi, _far(2))), dict(out=_rows(abi, _far(3))), dict(out=_rows(abi, _far(4)))):
        assert call(**bad) == abi.EINVAL, bad


def test_calls_without_rows_do_nothing(abi):
    """No rows: no pointer to rows is needed, nothing is launched."""
    L = abi.lib()
    null = lambda: C.byref(abi.kvd_rows(None, 0, 0))  # noqa: E731
    assert L.kv_paged_append_q8(None, null(), null(), 8, null(), null(), 8, 128, 0, 2, None, None, 0, _far(1), _far(2), _far(3), _far(4), 64, 16, FAKE, None) == abi.OK
    assert L.kv_paged_read(_far(1), _far(2), _far(3), _far(4), 3, 64, 16, 8, 128, FAKE, 8, FAKE, None, FAKE, 4, null(), null(), 2, 0, FAKE, None) == abi.OK
    assert L.paged_attention_q8(null(), null(), 0, 8, 8, 128, 2, _far(1), _far(2), _far(3), _far(4), 64, 16, FAKE, 8, FAKE, FAKE, 4, 0.1, 0, 0.0, None, None, 0, FAKE,
                                None) == abi.OK
