"""Products of more tiles than a launch holds are refused on the host, before
anything is launched."""
import pytest

from combine_routing_histogram_amd import binding as B
from combine_routing_histogram_amd import build as hip_build
from combine_routing_histogram_amd import layer as L

A = 1 << 44       # an aligned stand-in address: refused calls never touch it


@pytest.fixture(scope="module", autouse=True)
def lib():
    if hip_build.is_stale():
        hip_build.build()
    return L.lib()


def _args(rows, out, experts=1, activation=L.EPDC_ACT_NONE, **kw):
    return L.make_product_args(rows, experts, 8, out, activation=activation, input=A, weight=2 * A,
                               expert_off=3 * A, **kw)


# (arguments, block threads) with between 2^32 / threads and 2^31 blocks: whole
# tiles, 64-row tiles and the streamed form
TOO_MANY = [dict(rows=1 << 20, out=1 << 20),
            dict(rows=64 << 14, out=1 << 17, experts=512, expected_rows=64 * 512),
            dict(rows=1 << 17, out=1 << 16, experts=512, expected_rows=512)]


@pytest.mark.parametrize("kw", TOO_MANY)
def test_forward(kw):
    with pytest.raises(B.EpdcError) as ei:
        L.epdc_expert_product(_args(**kw), 0, 0, 4 * A, 0)
    assert ei.value.status == B.EPDC_ERR_INVALID_ARGS and "launch" in str(ei.value)


# rows' gradient, weights' gradient, and both, each of which alone would fit
@pytest.mark.parametrize("rows,experts,fin,fout,gx,gw", [
    (1 << 26, 1, 1 << 16, 8, 5 * A, 0), (1, 512, 1 << 20, 776, 0, 6 * A),
    (1 << 17, 512, 1 << 20, 520, 5 * A, 6 * A)])
def test_backward(rows, experts, fin, fout, gx, gw):
    args = L.make_product_args(rows, experts, fin, fout, input=A, weight=2 * A, expert_off=3 * A)
    with pytest.raises(B.EpdcError) as ei:
        L.epdc_expert_backward(args, 0, 4 * A, 0, 0, gx, gw, L.EPDC_DT_BF16, 0)
    assert ei.value.status == B.EPDC_ERR_INVALID_ARGS and "launch" in str(ei.value)


def test_backward_refuses_before_the_activation_is_launched():
    """A status other than SUCCESS leaves nothing enqueued: without a GPU the
    launch of the activation's gradient would show as another status."""
    args = L.make_product_args(1, 512, 1 << 20, 776, activation=L.EPDC_ACT_SILU, input=A,
                               weight=2 * A, expert_off=3 * A)
    with pytest.raises(B.EpdcError) as ei:
        L.epdc_expert_backward(args, 0, 4 * A, 8 * A, 9 * A, 0, 6 * A, L.EPDC_DT_BF16, 0)
    assert ei.value.status == B.EPDC_ERR_INVALID_ARGS and "tiles" in str(ei.value)
