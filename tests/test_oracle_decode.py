"""The decoding oracles without a GPU: the step against the chunked rule's oracle, the norm's
gradient against differences, attention against a hand-worked case."""
import numpy as np
import pytest

from chunked_prefill_gb300.inputs import make_inputs
from oracle import decode
from oracle import oracle as orc


@pytest.fixture(scope="module", autouse=True)
def _oracle():
    orc.build()


def test_step_continues_the_prefill():
    """A prefill of 40 tokens and 9 single steps give the outputs and state of 49 tokens."""
    inp = make_inputs(1, 49, 2, 4, seed=3, h0_std=0.2)
    o, ht = orc.fwd(inp.q, inp.k, inp.v, inp.g, inp.beta, inp.scale, h0=inp.h0)
    part = lambda t, a, b: t[:, a:b].contiguous()  # noqa: E731
    _, h = orc.fwd(*(part(t, 0, 40) for t in (inp.q, inp.k, inp.v, inp.g, inp.beta)), inp.scale, h0=inp.h0)
    for t in range(40, 49):
        x = [part(y, t, t + 1)[0].double().numpy() for y in (inp.q, inp.k, inp.v, inp.g, inp.beta)]
        ot, h = decode.step(*x, inp.scale, h, [0], [1])
        assert np.allclose(ot[0], o.reshape(49, 4, 128)[t], rtol=1e-9, atol=1e-12)
    assert np.allclose(h, ht, rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("offset,with_sum", [(0.0, False), (1.0, True)])
def test_norm_gradient_against_differences(offset, with_sum):
    rng = np.random.default_rng(5)
    s, dy, w = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7)
    ds = rng.normal(size=(3, 7)) if with_sum else None

    def loss(s, w):
        y, _ = decode.norm(s, w, eps=1e-3, offset=offset)
        return (y * dy).sum() + ((s * ds).sum() if with_sum else 0)

    dx, dw, _, _ = decode.norm_bwd(s, w, dy, ds, eps=1e-3, offset=offset)
    h = 1e-6
    for x, grad, at in ((s, dx, lambda z: loss(z, w)), (w, dw, lambda z: loss(s, z))):
        for i in np.ndindex(x.shape):
            up, down = x.copy(), x.copy()
            up[i] += h
            down[i] -= h
            # central differences: truncation ~ h^2, rounding ~ 1e-16 |loss| / h
            assert abs((at(up) - at(down)) / (2 * h) - grad[i]) < 1e-7


def test_paged_attention_by_hand():
    """Two tokens on two pages, one head: equal scores give the mean, a window of one the last."""
    k = np.zeros((3, 1, 1, 64))
    v = np.full((3, 1, 1, 64), np.nan)
    v[2], v[0] = 1.0, 3.0
    table = np.array([[2, 0]])
    o, lse, _, _ = decode.paged(np.ones((1, 1, 64)), k, v, table, [2], 0.5)
    assert np.allclose(o, 2.0) and np.allclose(lse, np.log(2))
    o, lse, _, _ = decode.paged(np.ones((1, 1, 64)), k, v, table, [2], 0.5, window=1)
    assert np.allclose(o, 3.0) and np.allclose(lse, 0.0)
    o, lse, _, _ = decode.paged(np.ones((1, 1, 64)), k, v, table, [0], 0.5)
    assert (o == 0).all() and (lse == -np.inf).all()
