"""The widest outputs of the linears with an epilogue, on the host: made-up addresses."""
import pytest
import torch

i8 = pytest.importorskip("int8_mixed_precision_rowwise_amd")
if torch.cuda.is_available():
    pytest.skip("addresses are made up: for hosts without a device", allow_module_level=True)

EINVAL, EDEVICE = 1, 3
G = 1 << 36


@pytest.mark.parametrize("N,status", [((1 << 28) - 1, EDEVICE), (1 << 28, EINVAL), ((1 << 28) + 1, EINVAL)])
def test_columns_past_one_launch_are_refused(N, status):
    """Past 2^32 work items a launch drops columns without a word."""
    ld = (N + 7) // 8 * 8
    p = i8._LinearAct(2, N, 16, G, 16, 2 * G, 16, 0, None, None, 0, 3 * G, ld, None, 0)
    assert i8.lib.i8mp_linear_act_fwd(p, i8._Opts(0, 0, 0), None, None, 4 * G, 1 << 40, None) == status
    assert i8.lib.i8mp_linear_wq_fwd(p, 5 * G, 16, 6 * G, None, 0, None) == status
    b = i8._LinearActGrad(2, N, 16, G, ld, None, 0, 2 * G, 16, None, 0, 0, None, 0, 3 * G, 16, 5 * G)
    assert i8.lib.i8mp_linear_act_bwd(b, i8._Opts(0, 0, 0), None, None, 7 * G, 1 << 50, None) == status
