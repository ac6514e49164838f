"""smoke() checks what it runs: it passes, and mistakes planted in its host references make it fail."""
import pytest

pytestmark = pytest.mark.gpu


def test_smoke_passes_and_runs_every_form(monkeypatch):
    import __graft_entry__ as entry
    from video_dit_mixed_gb300 import ops
    rows = {"grouped": set(), "few": set()}
    grouped, few = ops.qgemm_grouped, ops.qgemv
    monkeypatch.setattr(ops, "qgemm_grouped", lambda a, *r, **k: rows["grouped"].add(len(a.i8_codes)) or grouped(a, *r, **k))
    monkeypatch.setattr(ops, "qgemv", lambda a, *r, **k: rows["few"].add(len(a.i8_codes)) or few(a, *r, **k))
    entry.smoke()
    experts = 4
    assert any(m <= 8 for m in rows["grouped"])                       # dot products
    assert any(8 < m < 48 * experts for m in rows["grouped"])         # narrow token tiles
    assert any(m >= 48 * experts for m in rows["grouped"])            # wide ones
    assert any(m <= 2 for m in rows["few"]) and any(m > 2 for m in rows["few"])


def _off_by_one_code(ref):
    def wrong(codes, scales):
        v = ref(codes, scales)
        v[3] += scales.cpu().double()[0, 3]
        return v
    return wrong


@pytest.mark.parametrize("name,mistake,said", [
    ("_rms_norm", lambda f: lambda h: f(h) * 1.001, "norm scale parity"),
    ("_rotate", lambda f: lambda y, b: y, "norm scale parity"),
    ("_int4_values", _off_by_one_code, "few-row parity"),
    ("_experts_ref", lambda f: lambda *a, **k: f(*a, **k) * 1.02, "experts parity"),
])
def test_a_wrong_reference_is_noticed(monkeypatch, name, mistake, said):
    import __graft_entry__ as entry
    monkeypatch.setattr(entry, name, mistake(getattr(entry, name)))
    with pytest.raises(AssertionError, match=said):
        entry.smoke()
