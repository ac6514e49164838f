"""Argument checks, at the C boundary, of the calls around a feed-forward layer's products (host only: nothing is enqueued)."""
import ctypes as C

import pytest

EINVAL, ESHAPE, EALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from video_dit_mixed_gb300 import abi
    return abi.lib(build_if_missing=True)


@pytest.fixture()
def p():
    raw = C.create_string_buffer(4096)
    yield (C.addressof(raw) + 63) // 64 * 64
    del raw


def _expect(lib, call, *groups):
    before = lib.sixbit_launch_count()
    for want, cases in groups:
        for kw in cases:
            assert call(**kw) == want, kw
    assert lib.sixbit_launch_count() == before


def test_gated_rmsnorm_quant(lib, p):
    from video_dit_mixed_gb300 import abi

    def call(x=p, r=None, rs=1.0, w=None, post=None, gate=None, sc=None, sh=None, seg=None, s=1, m=2, k=128, eps=1e-6,
             b=16, h=None, y=None, codes=p, scale=p, out=True):
        qa = abi.QAct(None, None, None, None, codes, scale, None)
        return lib.sixbit_gated_rmsnorm_quant(x, r, rs, w, post, gate, sc, sh, seg, s, m, k, eps, b, None, h, y,
                                              C.byref(qa) if out else None, None, None)

    _expect(lib, call,
            (EINVAL, [dict(x=None), dict(codes=None), dict(scale=None), dict(eps=0.0), dict(eps=float("nan")),
                      dict(rs=float("inf")), dict(rs=float("nan")), dict(out=False), dict(y=p)]),
            (ESHAPE, [dict(m=-1), dict(k=0), dict(k=192), dict(k=16512), dict(b=32), dict(b=256), dict(s=0), dict(s=3)]),
            (EALIGN, [dict(x=p + 8), dict(r=p + 2), dict(w=p + 4), dict(post=p + 4), dict(gate=p + 8), dict(sc=p + 8),
                      dict(sh=p + 4), dict(seg=p + 2), dict(h=p + 8), dict(codes=p + 8), dict(scale=p + 2),
                      dict(y=p + 8, b=0)]),
            (0, [dict(m=0, x=None, codes=None, scale=None), dict(m=0, y=p, b=0, out=False)]))


def test_moe_route(lib, p):
    def call(l=p, lb=None, bias=None, t=2, e=8, k=2, score=0, groups=1, top=1, best=2, renorm=1, f=1.0, experts=p,
             w=p, rows=p, token=p, off=p, ws=None):
        return lib.sixbit_moe_route(l, lb, bias, t, e, k, score, groups, top, best, renorm, f, experts, w, rows, token,
                                    off, ws, None)

    _expect(lib, call,
            (ESHAPE, [dict(t=-1), dict(e=0), dict(e=1025), dict(k=0), dict(k=33, e=64), dict(k=9), dict(t=2**30, k=2),
                      dict(groups=0), dict(groups=3), dict(groups=33, e=66), dict(groups=4, top=0),
                      dict(groups=4, top=5), dict(groups=4, top=1, k=3)]),
            (EINVAL, [dict(score=2), dict(score=-1), dict(best=0), dict(best=3), dict(f=float("inf")), dict(l=None),
                      dict(experts=None), dict(w=None), dict(rows=None), dict(token=None), dict(off=None),
                      dict(t=33, ws=None), dict(t=0, off=None)]),
            (EALIGN, [dict(l=p + 2), dict(lb=p + 1), dict(bias=p + 2), dict(experts=p + 1), dict(w=p + 2),
                      dict(rows=p + 2), dict(token=p + 2), dict(off=p + 2), dict(ws=p + 8)]))
    assert lib.sixbit_moe_route_workspace_bytes(1, 8) == 0 and lib.sixbit_moe_route_workspace_bytes(0, 8) == 0
    assert lib.sixbit_moe_route_workspace_bytes(32, 8) == 0 and lib.sixbit_moe_route_workspace_bytes(33, 9) == 304 * 12 * 4


def test_moe_combine(lib, p):
    def call(d=p, df=None, rows=p, w=p, t=2, k=2, r=4, h=8, y=p, yf=None):
        return lib.sixbit_moe_combine(d, df, rows, w, t, k, r, h, y, yf, None, None)

    _expect(lib, call,
            (ESHAPE, [dict(t=-1), dict(k=0), dict(k=33), dict(r=-1), dict(h=0), dict(h=(1 << 20) + 1)]),
            (EINVAL, [dict(d=None), dict(rows=None), dict(w=None), dict(y=None)]),
            (EALIGN, [dict(d=p + 1), dict(df=p + 2), dict(rows=p + 2), dict(w=p + 2), dict(y=p + 1), dict(yf=p + 2)]),
            (0, [dict(t=0, d=None, rows=None, w=None, y=None)]))


def test_lowrank_add(lib, p):
    from video_dit_mixed_gb300 import abi

    def call(act=True, codes=p, scale=p, x=None, a=p, b=p, al=None, ids=p, l=2, m=2, n=16, k=128, r=16, base=None,
             bf=None, epi=0, res=None, y=p, yf=None, ws=p):
        qa = abi.QAct(None, None, None, None, codes, scale, None)
        return lib.sixbit_lowrank_add(C.byref(qa) if act else None, x, a, b, al, ids, l, m, n, k, r, base, bf, None, epi,
                                      res, y, yf, ws, None, None)

    _expect(lib, call,
            (ESHAPE, [dict(m=-1), dict(m=2**31 - 16), dict(n=0), dict(n=(1 << 20) + 1), dict(k=0), dict(k=64), dict(k=(1 << 20) + 128), dict(r=0),
                      dict(r=8), dict(r=24), dict(r=144), dict(l=0), dict(l=16385)]),
            (EINVAL, [dict(act=False), dict(codes=None), dict(scale=None), dict(a=None), dict(b=None), dict(ids=None),
                      dict(y=None), dict(m=129, ws=None), dict(epi=2), dict(epi=3), dict(epi=-1), dict(base=p, bf=p)]),
            (EALIGN, [dict(codes=p + 8), dict(scale=p + 2), dict(x=p + 8), dict(a=p + 8), dict(b=p + 4), dict(al=p + 2),
                      dict(ids=p + 2), dict(base=p + 1), dict(bf=p + 2), dict(epi=2, res=p + 1), dict(y=p + 1),
                      dict(yf=p + 2), dict(ws=p + 8)]),
            (0, [dict(m=0, act=False, a=None, b=None, ids=None, y=None, ws=None)]))
    for r, few in ((32, 128), (48, 64)):  # what the binding allocates
        for m in (0, 1, few, few + 1, 1001):
            assert lib.sixbit_lowrank_workspace_bytes(m, r) == (0 if m <= few else m * r * 6 + 2 * ((4 * m + 15) // 16 * 16))
