"""A scale that fp32 cannot hold is refused (no GPU needed)."""
import pytest

from test_layer_abi_host import CALLS, INVALID, lib, lib_call, put_all  # noqa: F401


@pytest.mark.parametrize("value", [1e39, -1e300])
@pytest.mark.parametrize("name,field", [("delta", "scale"), ("delta_bwd", "fwd.scale"), ("delta_step", "scale")])
def test_scales_past_fp32(name, field, value):
    assert lib_call(name, put_all(CALLS[name](), {field: value})) == INVALID
