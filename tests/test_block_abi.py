"""Host-only checks of include/ttc_block.h: descriptors are validated, sizes
queried and argument errors returned before anything is launched.  No GPU."""

import pytest

import tensor_train_compressed_tt_amd as ttc


def _code(f, *a):
    with pytest.raises(ttc.TTCError) as e:
        f(*a)
    return e.value.code


@pytest.mark.parametrize("kw,code", [(dict(n=0), 2), (dict(n=(1 << 20) + 1), 2), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
                                     (dict(x_dtype=ttc.TTC_FP8), 4), (dict(x_dtype=9), 4), (dict(y_dtype=-1), 4)])
def test_norm_descriptors(kw, code):
    d = ttc.make_norm_desc(**{"n": 768, **kw})
    assert _code(ttc.ttc_norm_workspace, d, 64) == code


def test_norm_sizes():
    d = ttc.make_norm_desc(768, ttc.TTC_BF16, ttc.TTC_BF16)
    assert ttc.ttc_norm_workspace(d, 0) == (0, 0)
    s, c = ttc.ttc_norm_workspace(d, 16384)
    assert s == 16384 * 8 and c == 256 * 2 * 768 * 4
    assert _code(ttc.ttc_norm_workspace, d, -1) == 2
    assert _code(ttc.ttc_norm_workspace, d, 1 << 31) == 2


def test_norm_errors_before_launch():
    d = ttc.make_norm_desc(768, ttc.TTC_BF16, ttc.TTC_BF16)
    s, c = ttc.ttc_norm_workspace(d, 64)
    fwd = dict(x=16, res=16, gamma=16, beta=16, h=16, y=16, saved=16, saved_bytes=s)
    call = lambda **kw: ttc.ttc_norm_fwd(d, 64, **{**fwd, **kw})  # noqa: E731
    for k in ("x", "gamma", "beta", "h", "y", "saved"):
        assert _code(lambda: call(**{k: None})) == 1, k
        assert _code(lambda: call(**{k: 24})) == 5, k
    assert _code(lambda: call(saved_bytes=s - 1)) == 6
    bwd = dict(dy=16, h=16, gamma=16, dh=None, saved=16, saved_bytes=s, dx=16, dgamma=16, dbeta=16, scratch=16, scratch_bytes=c)
    call = lambda **kw: ttc.ttc_norm_bwd(d, 64, **{**bwd, **kw})  # noqa: E731
    for k in ("dy", "h", "gamma", "saved", "dx", "dgamma", "dbeta", "scratch"):
        assert _code(lambda: call(**{k: None})) == 1, k
        assert _code(lambda: call(**{k: 24})) == 5, k
    assert _code(lambda: call(dh=8)) == 5
    assert _code(lambda: call(saved_bytes=s - 1)) == 6 and _code(lambda: call(scratch_bytes=c - 1)) == 6
    ttc.ttc_norm_fwd(d, 0, None, None, None, None, None, None, None, 0)  # no rows: nothing is touched
