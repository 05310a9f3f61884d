"""Outputs in the place of inputs at another row distance are refused before anything is launched (no GPU
needed)."""
import pytest

from test_block_abi import NORM, P, QUANT, ROTARY, _status, r  # noqa: F401

LD = dict(ldx=256, ldr=512, ldh=264)


@pytest.mark.parametrize("kw", [
    dict(LD, X=P, R=2 * P, H=P, Y=4 * P), dict(LD, X=3 * P, R=P, H=P, Y=4 * P),
    dict(LD, X=P, R=2 * P, H=3 * P, Y=P, ldy=272), dict(LD, X=P, R=2 * P, H=3 * P, Y=2 * P, ldy=256),
    dict(X=P, R=None, H=None, Y=P, ldx=256, ldy=264),
])
def test_norm(r, kw):  # noqa: F811
    assert _status(r, "rudder_norm", NORM, kw) == 1
    assert "elements apart" in r.load_library().rudder_last_error().decode()


@pytest.mark.parametrize("kw", [dict(LD, X=P, R=2 * P, H=P), dict(LD, X=3 * P, R=P, H=P)])
def test_norm_quant(r, kw):  # noqa: F811
    assert _status(r, "rudder_norm_quant", QUANT, kw) == 1
    assert "elements apart" in r.load_library().rudder_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(Q=P, Qo=P, ldq=512, ldqo=256, K=2 * P, Ko=3 * P),
    dict(Q=P, Qo=2 * P, K=3 * P, Ko=3 * P, ldk=512, ldko=128),
])
def test_rotary(r, kw):  # noqa: F811
    assert _status(r, "rudder_rotary", ROTARY, kw) == 1
    assert "elements apart" in r.load_library().rudder_last_error().decode()
