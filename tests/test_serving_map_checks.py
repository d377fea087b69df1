"""dmoe_mx4_forward refuses a map that was not made for the call's sizes and kind of routing; on the
host, nothing is launched."""
import pytest

from dropless_mixture_experts_dmoe_b200 import binding as B

FAKE = 1 << 20


@pytest.fixture(scope="module")
def weights():
    q = B.Mx4.empty(8, 128, 256, device="cpu")
    return q, q, B.Mx4.empty(8, 256, 128, device="cpu")


def call(dims, w, smap):
    B.dmoe_mx4_forward(dims, FAKE, *w, smap, FAKE, FAKE)


@pytest.mark.parametrize("field,value", [("T", 5), ("hidden", 384), ("num_experts", 4),
                                         ("top_k", 1)])
def test_sizes_changed_after_the_map(weights, field, value):
    """The same object, changed since: the map keeps what it was made for."""
    d = B.make_dims(4, 256, 128, 8, 2)
    m = B.Mx4Buffers(d, device="cpu")
    setattr(d, field, value)
    with pytest.raises(ValueError, match="the map is"):
        call(d, weights, m.map)


@pytest.mark.parametrize("made,asked", [(B.ROUTE_TOKEN_ROUNDING, 0), (0, B.ROUTE_TOKEN_ROUNDING)])
def test_kind_of_entry_list(weights, made, asked):
    """With token rounding the map is an entry list of another length and order."""
    m = B.Mx4Buffers(B.make_dims(200, 256, 128, 8, 2, flags=made), device="cpu")
    with pytest.raises(ValueError, match="the map is"):
        call(B.make_dims(200, 256, 128, 8, 2, flags=asked), weights, m.map)


def test_flags_that_do_not_matter(weights):
    """Flags that choose between forms of other calls: refused for the device alone."""
    m = B.Mx4Buffers(B.make_dims(200, 256, 128, 8, 2, flags=B.SAVE_X_ONLY), device="cpu")
    with pytest.raises(ValueError, match="smap.status"):
        call(B.make_dims(200, 256, 128, 8, 2, flags=B.FUSED_COMBINE | B.ROUTE_RENORMALIZE), weights,
             m.map)
