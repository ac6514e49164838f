"""Argument checks of the feed-forward calls at the C boundary (host only: nothing is enqueued)."""
import ctypes as C

import pytest

EINVAL, ESHAPE, EALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from video_dit_mixed_gb300 import abi
    return abi.lib(build_if_missing=True)


@pytest.fixture()
def buf():
    raw = C.create_string_buffer(4096)
    at = (C.addressof(raw) + 63) // 64 * 64
    return raw, at


def test_add_rmsnorm_quant(lib, buf):
    from video_dit_mixed_gb300 import abi
    _, p = buf
    before = lib.sixbit_launch_count()

    def call(x=p, r=None, w=None, m=2, k=128, eps=1e-6, b=16, h=None, codes=p, scale=p):
        qa = abi.QAct(None, None, None, None, codes, scale, None)
        return lib.sixbit_add_rmsnorm_quant(x, r, w, m, k, eps, b, None, h, C.byref(qa), None, None)

    for kw in (dict(x=None), dict(codes=None), dict(scale=None), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")),
               dict(eps=float("nan")), dict(h=p)):
        assert call(**kw) == EINVAL, kw
    for kw in (dict(m=-1), dict(k=0), dict(k=192), dict(b=32), dict(b=256), dict(b=-16)):
        assert call(**kw) == ESHAPE, kw
    for kw in (dict(x=p + 8), dict(r=p + 2), dict(w=p + 4), dict(r=p, h=p + 8), dict(codes=p + 8), dict(scale=p + 2)):
        assert call(**kw) == EALIGN, kw
    assert call(m=0, x=None, codes=None, scale=None) == 0
    assert lib.sixbit_add_rmsnorm_quant(p, None, None, 2, 128, 1e-6, 16, None, None, None, None, None) == EINVAL
    assert lib.sixbit_launch_count() == before


@pytest.mark.parametrize("grouped", [False, True])
def test_products(lib, buf, grouped):
    from video_dit_mixed_gb300 import abi
    _, p = buf
    before = lib.sixbit_launch_count()

    def call(m=2, n=16, k=128, epi=0, res=None, y=p, yf=None, codes=p, scale=p, w4=p, ws=p, off=p, e=2, work=p,
             a=True, w=True):
        qa = abi.QAct(None, None, None, None, codes, scale, None)
        qw = abi.Weights(None, None, None, None, w4, ws, None)
        ca, cw = C.byref(qa) if a else None, C.byref(qw) if w else None
        if grouped:
            return lib.sixbit_qgemm_grouped(ca, cw, off, e, m, n, k, None, epi, res, y, yf, work, None, None)
        return lib.sixbit_qgemv(ca, cw, m, n, k, None, epi, res, y, yf, None, None)

    bad = [dict(a=False), dict(w=False), dict(codes=None), dict(scale=None), dict(w4=None), dict(ws=None),
           dict(y=None), dict(epi=3), dict(epi=-1), dict(epi=2)]
    shape = [dict(m=-1), dict(n=0), dict(k=0), dict(k=64)]
    align = [dict(codes=p + 8), dict(w4=p + 4), dict(scale=p + 2), dict(ws=p + 1), dict(epi=2, res=p + 1),
             dict(y=p + 1), dict(yf=p + 2)]
    if grouped:
        shape += [dict(e=0), dict(e=1025)]
        align += [dict(off=p + 2)]
    else:
        shape += [dict(m=33)]
    for want, cases in ((EINVAL, bad), (ESHAPE, shape), (EALIGN, align)):
        for kw in cases:
            assert call(**kw) == want, kw
    assert call(m=0, codes=None, scale=None, y=None) == 0
    assert lib.sixbit_launch_count() == before
    assert lib.sixbit_qgemm_grouped_workspace_bytes(35552, 12288) == 35552 * 12288 * 2 + 35552 * 96 * 4
    assert lib.sixbit_qgemm_grouped_workspace_bytes(0, 128) == 0
