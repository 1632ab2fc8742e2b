"""Arguments of the wrong kind to the operators on packed sequences: an error that names
them, from every entry point that takes them, with nothing written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_wrong_kinds_are_named():
    import selective_state_space_38_b200 as ssm
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    cu, win = torch.tensor([0, 4], dtype=torch.int32, device="cuda"), torch.zeros(4, 3, 8, device="cuda")
    h = dict(x=torch.zeros(4, 2, 64, device="cuda"), dt=torch.zeros(4, 2, device="cuda"), A=torch.zeros(2, device="cuda"),
             B=torch.zeros(4, 1, 128, device="cuda"))
    step = lambda st: ssm.ssm_ssd_step(st, h["x"], h["dt"], None, True, h["A"], h["B"], h["B"])  # noqa: E731
    packed = lambda **kw: ssm.ssm_ssd_varlen_fwd(  # noqa: E731
        h["x"].bfloat16(), h["dt"].bfloat16(), None, True, h["A"], h["B"].bfloat16(), h["B"].bfloat16(), None, cu, **kw)
    for name, kind, call in (
            ("has_initial", TypeError, lambda: ssm.ssm_conv1d_fwd(x, w, None, cu, windows=win, has_initial=[True])),
            ("has_initial", TypeError, lambda: packed(has_initial=[True])),
            ("conv_w", TypeError, lambda: ssm.ssm_conv1d_fwd(x, [[0.0] * 4] * 8, None, cu)),
            ("conv_w", ValueError, lambda: ssm.ssm_conv1d_fwd(x, w[:, None], None, cu)),
            ("conv_w", ValueError, lambda: ssm.ssm_conv1d_bwd(x, w[0], None, cu, x)),
            ("conv_w", ValueError, lambda: ssm.ssm_conv1d_step(win, x, w[0], None)),
            ("windows", TypeError, lambda: ssm.ssm_conv1d_fwd(x, w, None, cu, windows=[0.0])),
            ("windows", ValueError, lambda: ssm.ssm_conv1d_step(win[0], x, w, None)),
            ("states", TypeError, lambda: packed(states=[0.0])),
            ("states", ValueError, lambda: packed(states=win)),
            ("states", TypeError, lambda: step(None)),
            ("states", ValueError, lambda: step(win))):
        with pytest.raises(kind, match=name):
            call()
