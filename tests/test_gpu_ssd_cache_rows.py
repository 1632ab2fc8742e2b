"""The packed SSD where every sequence goes on from its cache row and leaves its state
there, in each of the three schedules with all SMs busy, against float64 and call after
call.  The layouts of the two passes put sequences' first segments behind others in a
CTA's work list while their last ones, of a step or two, come up elsewhere."""
import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
RANGES, TWO_PASSES, CHAINS = 0, 1, 2


def _expected(inp, lens, states, slots):
    """(y, states, the same of the terms' magnitudes) in float64, every sequence from its cache row."""
    d = {k: v.cuda().double() for k, v in inp.items()}
    dt, at = ref.softplus(d["dt"] + d["dt_bias"]), ref.offsets(lens)
    res = []
    for f in (lambda v: v, torch.abs):
        x, B, C, D = (f(d[k]) for k in ("x", "B", "C", "D"))
        y, st = torch.empty_like(x), f(states.cuda().double())
        for i, slot in enumerate(slots.tolist()):
            r = slice(at[i], at[i + 1])
            y[r], st[slot] = ref.ssd_sequence(x[r], dt[r], d["A"], B[r], C[r], D, st[slot])
        res += [y.cpu(), st.cpu()]
    return res


@pytest.mark.parametrize("H,lens,schedule", [
    (24, [8192] * 2 + [1] * 10 + [641] * 4, TWO_PASSES),
    (24, [1024], TWO_PASSES),
    (6, [257] * 40 + [6000], TWO_PASSES),
    (24, [1500] * 10, CHAINS),
    (24, [50, 1300, 128, 700] * 8, RANGES),
])
def test_sequences_that_go_on_and_end_in_one_cache_row(H, lens, schedule):
    import selective_state_space_38_b200 as ssm
    g = ref.gen(H + len(lens))
    inp, n = ref.ssd_inputs(g, sum(lens), H, 1), len(lens)
    states = ref.randn(g, n + 1, H, 64, 128)
    slots = torch.randperm(n + 1, generator=g)[:n].to(torch.int32)
    d = {k: v.cuda() for k, v in inp.items()}
    cu = torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")
    workspace = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(4):
        st = states.cuda()
        y = ssm.ssm_ssd_varlen_fwd(d["x"], d["dt"], d["dt_bias"], True, d["A"], d["B"], d["C"], d["D"], cu, states=st,
                                   slots=slots.cuda(), has_initial=torch.ones(n, dtype=torch.bool, device="cuda"),
                                   workspace=workspace, check=True)
        assert int(workspace[28:32].view(torch.int32)) == schedule
        if first is None:
            first = (y, st)
        assert torch.equal(y, first[0]) and torch.equal(st, first[1])
    ry, rst, ay, ast = _expected(inp, lens, states, slots)
    ref.close(first[0], ry, ref.ssd_y_tolerance(ry, ay), "y")
    ref.close(first[1], rst, ref.ssd_state_tolerance(ast, max(lens) // 128 + 2), "states")
