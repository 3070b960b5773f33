"""Without a GPU: refusals at the ends of the layer operators' ranges (on the host, before anything is launched)."""
import pytest

from test_layer_ops_cpu import lib, rot, view  # noqa: F401


@pytest.mark.parametrize("grid,start,code", [((1, 1), 2 ** 31 - 4, 0), ((1, 1), 2 ** 31 - 3, -1), ((1, 1), 2 ** 52, -1),
                                             ((64, 128), 2 ** 44 - 4, 0), ((64, 128), 2 ** 44 - 3, -1), ((64, 128), 2 ** 52, -1)])
def test_rotary_refuses_frames_beyond_int32(lib, grid, start, code):
    """A grid's positions end where int32 positions do: the angles of farther ones have no accuracy left.  (The accepted calls
    end at the next check, of q's data.)"""
    got = rot(lib, gh=grid[0], gw=grid[1], start=start, q=view(0))
    assert got == -1 and (b"frame" in lib.gdn_last_error()) == (code != 0)
    assert code or b"q must be" in lib.gdn_last_error()


def test_a_stream_of_another_device_is_refused():
    """torch.cuda.stream makes the stream's device current: the kernels would run there, on pointers of the tensors' device."""
    import types

    import torch
    from gated_delta_rule_149_b200.gdn import _run

    def call(handle):
        raise AssertionError("called")

    with pytest.raises(ValueError, match="stream"):
        _run(torch.device("cuda", 0), types.SimpleNamespace(device=torch.device("cuda", 1)), call)
