"""What a call reads of an argument's attributes stays alive until the call is over
(no GPU: the calls here are refused at their last argument)."""
import weakref

import pytest

from test_ops_binding import BF, bsq, on  # noqa: F401 (bsq: the fixture)
from test_more_ops_abi import D, N, T, U8


class Made:
    """A quantized tensor that makes its buffers when it is asked for them"""
    fmt, tensor_scale = 0, None

    def __init__(self, rows, seen, before=()):
        self.rows, self.cols, self.seen, self.before = rows, D, seen, before

    def make(self, n):
        t = on(0, n, dtype=U8)
        self.seen.append(weakref.ref(t))
        return t

    @property
    def codes(self):
        assert all(r() is not None for r in self.before), "buffers of an operand before this one are gone"
        return self.make(self.rows * self.cols)

    @property
    def scales(self):
        assert all(r() is not None for r in self.before), "buffers of an operand before this one are gone"
        return self.make(512 * -(-self.rows // 128) * -(-self.cols // 128))


def test_buffers_of_quantized_operands(bsq):  # noqa: F811
    # (`before` is the list that fills while the call reads the operand before)
    a, b = [], []
    first, second, third = Made(T, a), Made(N, b, a), Made(N, [], a)
    bad = on(0, T, N + 1, dtype=BF)
    with pytest.raises(bsq.BsqError, match="not 4 x 24"):
        bsq.gemm_linear_into(first, second, bad)
    assert len(a) == 2 and len(b) == 2 and all(r() is None for r in a + b)
    a.clear()
    with pytest.raises(bsq.BsqError, match="not 4 x 24"):
        bsq.gemm_gated_into(first, second, third, bad)
    assert len(a) == 2
