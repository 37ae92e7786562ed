"""The binding's device checks of the 8-bit calls, with stand-ins for tensors (no GPU)."""
import pytest


class On:
    """What the checks look at of a tensor on a device."""

    def __init__(self, device, shape=(4, 64)):
        self.device, self.shape = f"cuda:{device}", shape
        self.index = device

    def get_device(self):
        return self.index


class Holder:
    def __init__(self, **kw):
        self.__dict__.update(kw)


@pytest.fixture(scope="module")
def sb():
    from video_diffusion_mixed_b200 import sixbit
    return sixbit


def test_a_workspace_on_another_device_is_refused(sb):
    ws = Holder(buf=On(1))
    with pytest.raises(sb.SixbitError, match="expected cuda:0") as e:
        sb.fp8_encode(On(0), Holder(codes=On(0)), ws)
    assert e.value.status == sb.SB_EINVAL
    with pytest.raises(sb.SixbitError, match="expected cuda:0"):
        sb.WeightFp8(On(0), None, ws)
    with pytest.raises(sb.SixbitError, match="expected cuda:0"):
        sb.linear_fp8(None, Holder(rows=4, codes=On(0)), Holder(w=Holder(codes=On(0)), K=64, N=32), On(0), ws=ws)
