"""How far the angles of pa_rope_init's speeds are from the formula's, against 60 decimal digits.

theta^(-2i / R) is a double's power: its exponent carries one rounding, which its
logarithm y = 2i / R ln(theta) magnifies, the power is off by less than two units of 2^-53,
the division by 2 pi (a rounded constant) by two more. So a speed of f / (2 pi) turns is off by at most
e^-y (y + 4) / (2 pi) 2^-53 <= 4 / (2 pi) 2^-53, and 2^-64 of it is cut off: below 2^-53 of a
turn for each position. Position times speed modulo 2^64 adds nothing."""
from decimal import Decimal, localcontext

import pytest

N = pytest.importorskip("paged_kv_cache_270_gb300._native")

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_270_gb300 import build
    build.build()


@pytest.mark.parametrize("theta", [2.0, 10000.0, 500000.0, 1e8])
@pytest.mark.parametrize("rot", [2, 20, 64, 128])
def test_angles_at_far_positions(theta, rot):
    rope = N.pa_rope_init(N.pa_rope_desc(N.PA_ROPE_HALF, rot, N.PA_ROPE_SCALE_NONE, theta, 1.0, 8192.0, 1.0, 4.0, 1.0))
    with localcontext() as ctx:
        ctx.prec = 60
        for i in range(rot // 2):
            speed = (Decimal(theta).ln() * (Decimal(-2 * i) / Decimal(rot))).exp() / (2 * PI)
            for p in (1, 1000, 1 << 20, (1 << 31) - 1, -12345, -(1 << 31)):
                got = Decimal(rope.step[i] * p % (1 << 64)) / (1 << 64)
                off = (got - speed * p) % 1
                off = min(abs(off), abs(1 - abs(off)))
                assert off <= abs(p) * Decimal(2) ** -53, (i, p, off)
