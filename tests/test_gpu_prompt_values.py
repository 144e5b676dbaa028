"""prompt_attention where a value, or every score, that a row sees is not finite."""
import math

import pytest
import torch

from tests.test_gpu_prompt import cu_of, normal

pytestmark = pytest.mark.gpu

DIMS = [(2, 1, 64, 64), (2, 1, 128, 128), (2, 1, 80, 40), (1, 1, 192, 128), (1, 1, 192, 192), (1, 1, 256, 256)]


@pytest.fixture(scope="module")
def nvm():
    import nvfp4_w4a16_mtp_amd as nv
    return nv


def inputs(seed, n, hq, hk, dk, dv):
    gen = torch.Generator().manual_seed(seed)
    return normal(gen, n, hq, dk), normal(gen, n, hk, dk), normal(gen, n, hk, dv)


@pytest.mark.parametrize("hq,hk,dk,dv", DIMS)
@pytest.mark.parametrize("place", ["below", "before a climb", "above"])
@pytest.mark.parametrize("t", [0, 40, 150])
def test_a_value_that_is_seen_counts_whatever_its_weight(nvm, hq, hk, dk, dv, place, t):
    """Weights are positive, so an infinite value is the average's and a NaN too: where its token's
    score lies 2^-400 below the others, where the row's reference moves by as much after it, and
    where it has all the weight; in tiles that all rows see and in those that some see."""
    n = 470
    q, k, v = inputs(t, n, hq, hk, dk, dv)
    q[:, :, 0] = 16.0
    k[:, :, 0] = 0.0
    step = 25.0 * math.sqrt(dk)                       # scores 400 apart, times log2(e)
    if place == "below":
        k[t, :, 0] = -step
    elif place == "above":
        k[t, :, 0] = step
    else:
        k[200:, :, 0] = step
    clean = nvm.prompt_attention(q, k, v, cu_of([n]), n)
    for bad in ((math.inf,), (-math.inf,), (math.nan,), (math.inf, -math.inf)):
        w = v.clone()
        for i, x in enumerate(bad):
            w[t + i, :, 1] = x
        y = nvm.prompt_attention(q, k, w, cu_of([n]), n)
        other = [d for d in range(dv) if d != 1]
        assert torch.equal(y[:, :, other], clean[:, :, other])
        assert torch.equal(y[:t], clean[:t])
        last = y[t + len(bad) - 1:, :, 1]
        assert bool((last.isnan() if len(bad) > 1 or math.isnan(bad[0]) else last == bad[0]).all()), (bad, last)
        if len(bad) > 1:
            assert bool((y[t, :, 1] == bad[0]).all())


@pytest.mark.parametrize("hq,hk,dk,dv", DIMS)
def test_infinities_beside_sums_past_fp32(nvm, hq, hk, dk, dv):
    """The largest finite values, whose sum has to be made again with smaller weights, and an infinity far back."""
    n = 300
    q, k, v = inputs(3, n, hq, hk, dk, dv)
    top = torch.finfo(torch.bfloat16).max
    v[:] = top
    v[7, :, 2] = -math.inf
    y = nvm.prompt_attention(q, k, v, cu_of([n]), n)
    other = [d for d in range(dv) if d != 2]
    assert bool((y[:, :, other] == top).all()) and bool((y[:7] == top).all()) and bool((y[7:, :, 2] == -math.inf).all())


@pytest.mark.parametrize("hq,hk,dk,dv", DIMS)
@pytest.mark.parametrize("how", ["k", "q", "range"])
def test_rows_without_a_score_above_minus_infinity(nvm, hq, hk, dk, dv, how):
    """No softmax: NaN.  Beside one finite score the others have no weight."""
    n = 200
    q, k, v = inputs(4, n, hq, hk, dk, dv)
    q[:], k[:] = 0.0, 0.0
    q[:, :, 0], k[:, :, 0] = 1.0, -1.0
    if how == "k":
        k[:, :, 0] = -math.inf
    elif how == "q":
        q[:, :, 0] = math.inf
    else:
        q[:, :, 0], k[:, :, 0] = 2.0 ** 70, -2.0 ** 70
    y = nvm.prompt_attention(q, k, v, cu_of([n]), n)
    assert bool(y.isnan().all())
    if how != "q":
        k[70, :, 0] = 0.0
        y = nvm.prompt_attention(q, k, v, cu_of([n]), n)
        want = v[70].repeat_interleave(hq // hk, 0)
        assert bool(y[:70].isnan().all()) and bool((y[70:] == want).all())


def test_a_score_of_infinity(nvm):
    q, k, v = inputs(5, 200, 2, 1, 128, 128)
    q[:, :, 0] = q[:, :, 0].abs() + 1.0
    q[60, :, 0] = -q[60, :, 0]
    clean = nvm.prompt_attention(q, k, v, cu_of([200]), 200)
    k[50, :, 0] = math.inf
    y = nvm.prompt_attention(q, k, v, cu_of([200]), 200)
    assert torch.equal(y[:50], clean[:50]) and bool(y[50:60].isnan().all()) and bool(y[61:].isnan().all())
    assert bool(y[60].isfinite().all())               # (its score is -inf)
