"""Token sampling without a GPU: every refusal of the entry point, which comes before any device
memory is touched (the addresses are fake), and the tests' own 64-bit form on rows worked out by
hand."""
import math
import os

import numpy as np
import pytest

import sample_ref as R

bd = pytest.importorskip("tenant_serving_bitdelta_amd")
if not os.path.exists(bd.LIB_PATH):
    pytest.skip("libbitdelta.so not built", allow_module_level=True)

L = bd.lib()
OK, INVALID, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 5
FAKE = 0x7F0000000000


def _call(logits=FAKE, dtype=1, rows=4, vocab=100, stride=100, u=FAKE, temp=FAKE, k=FAKE, p=FAKE,
          m=FAKE, tokens=FAKE, logprob=FAKE):
    return L.bitdelta_sample(logits, dtype, rows, vocab, stride, u, temp, k, p, m, tokens, logprob,
                             None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(tokens=None), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(vocab=0), INVALID), (dict(stride=99), SHAPE), (dict(logits=FAKE + 2), ALIGN),
    (dict(dtype=0, logits=FAKE + 1), ALIGN), (dict(u=FAKE + 2), ALIGN), (dict(temp=FAKE + 1), ALIGN),
    (dict(k=FAKE + 2), ALIGN), (dict(p=FAKE + 3), ALIGN), (dict(m=FAKE + 2), ALIGN),
    (dict(tokens=FAKE + 2), ALIGN), (dict(logprob=FAKE + 2), ALIGN),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), UNSUPPORTED), (dict(rows=(1 << 30) + 1), UNSUPPORTED),
])
def test_refusals(kw, status):
    assert _call(**kw) == status


def test_no_rows_is_a_no_op():
    assert _call(rows=0, logits=None, u=None, tokens=None) == OK


def test_reference_by_hand():
    ln = math.log
    row = np.array([ln(1), ln(4), -np.inf, ln(4), ln(1)])  # order: 1, 3, 0, 4 (weights 4 4 1 1 / 4)
    draw = lambda u, **kw: R.sample_row(row, u, **kw)
    assert [draw(u)[0] for u in (0.0, 0.39, 0.41, 0.79, 0.81, 0.89, 0.91)] == [1, 1, 3, 3, 0, 0, 4]
    assert draw(0.999, k=3)[0] == 0 and draw(0.999, k=2)[0] == 3 and draw(0.999, k=1)[0] == 1
    assert draw(0.999, p=0.5)[0] == 3 and draw(0.999, p=0.3)[0] == 1 and draw(0.999, p=0.85)[0] == 0
    assert draw(0.999, m=0.3)[0] == 3 and draw(0.999, m=0.2)[0] == 4 and draw(0.999, m=2.0)[0] == 1
    # top-p counts the first k's weight: 4/9 < 0.6 <= 8/9
    assert draw(0.999, k=3, p=0.6)[0] == 3
    assert draw(0.9, t=0.0) == (1, 0.0)
    assert abs(draw(0.5)[1] - ln(0.4)) < 1e-12
    assert R.sample_row(np.full(3, -np.inf), 0.5) == (-1, -np.inf)
