"""The packed SSD at the magnitudes of its operands: it is linear in (x, states), in B
with the states and in C, so operands of other scales give other scales of the same
results, whatever the decays within a chunk are."""
import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
LENS = [260, 140]


def _inputs(rates, seed=41):
    """Two heads that decay by these rates a step, the second sequence's steps varying fourfold."""
    inp = ref.ssd_inputs(ref.gen(seed), sum(LENS), 2, 1)
    steps = torch.full((sum(LENS), 2), 0.1)
    steps[260:] = 0.05 + 0.15 * torch.rand(140, 2, generator=ref.gen(seed + 1))
    inp.update(dt=torch.log(torch.expm1(steps)).to(torch.bfloat16), dt_bias=None, D=None, A=torch.tensor([-10.0 * r for r in rates]))
    return inp, ref.randn(ref.gen(seed + 2), 2, 2, 64, 128)


def _call(inp, states):
    import selective_state_space_38_b200 as ssm
    d, st = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in inp.items()}, states.cuda()
    cu = torch.tensor(ref.offsets(LENS), dtype=torch.int32, device="cuda")
    y = ssm.ssm_ssd_varlen_fwd(d["x"], d["dt"], None, True, d["A"], d["B"], d["C"], None, cu, states=st,
                               has_initial=torch.tensor([True, True], device="cuda"), check=True)
    return y, st


# 128 steps of 0.3 span e^38, of 0.53 e^68 and of 0.56 e^72, about the limit of factors by columns; of 1 and 4 they
# need the other two forms.
@pytest.mark.parametrize("rates", [(0.01, 0.3), (0.53, 0.56), (1.0, 0.02), (4.0, 1.0)])
@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 40])
@pytest.mark.parametrize("which", ["x", "B", "B and C"])
def test_operands_times_powers_of_two(rates, scale, which):
    """The results are those of the operands of order 1, times the power, within the bounds of the roundings.  With
    factors between e^-35 and e^35 = 2^51, the formats' 2^-126 to 2^127 leave 2^-75 to 2^76 for the operands, their
    steps and the lengths of the sums."""
    inp, states = _inputs(rates)
    half = 2.0 ** (20 if scale > 1 else -20)
    by = {"x": dict(x=scale), "B": dict(B=scale), "B and C": dict(B=half, C=half)}[which]
    of_state = by.get("x", 1.0) * by.get("B", 1.0)
    y, st = _call(dict(inp, **{k: inp[k] * v for k, v in by.items()}), states * of_state)
    ry, rst = ref.ssd(inp, LENS, states, None, [True, True])
    ay, ast = ref.ssd(inp, LENS, states, None, [True, True], absolute=True)
    ref.close(y.cpu().double() / scale, ry, ref.ssd_y_tolerance(ry, ay), "y")
    ref.close(st.cpu().double() / of_state, rst, ref.ssd_state_tolerance(ast, 4), "states")


@pytest.mark.parametrize("rate", [0.3, 0.54, 0.56, 1.0, 4.0])
@pytest.mark.parametrize("size", [1e-18, 1e-11, 1.0, 1e18])
def test_states_alone(rate, size):
    """x is zero: y is what is left of the states before, small or large, relative to its own size."""
    inp, states = _inputs((rate, 0.9 * rate))
    inp["x"].zero_()
    states = states * size
    y, st = _call(inp, states)
    ry, rst = ref.ssd(inp, LENS, states, None, [True, True])
    ay, ast = ref.ssd(inp, LENS, states, None, [True, True], absolute=True)
    dt, at = ref.softplus(inp["dt"].double()), ref.offsets(LENS)
    cs = torch.cat([(dt[i:j] * inp["A"].double()).cumsum(0) for i, j in zip(at, at[1:])])  # from the sequence's start
    # an exponent is a sum in float32 (16 roundings of 2^-24 deep, softplus and the product among them)
    drift = cs.abs() * 2.0 ** -20
    # results below the normal values: their absolute steps, 128 products in a sum; and a row whose decay passes e^-70
    # within a chunk feels that much of the state (128 products of at most 8 x 8)
    tiny, gone = 2.0 ** -120, (cs < -69.0) * (2.0 ** -100 * 128 * 64 * size)
    # The state meets C as a bf16 operand s = f S, and the row's factor r takes f back: r <= e^35 < 2^51.  An s below
    # 2^-126 is a subnormal or zero, off by at most 2^-126 itself; so y is off by r sum_n 2^-126 |C_n| <= 2^-75 sum |C_n|.
    # (A state that has decayed to 2^-75 within the chunks before is such a case, whatever its size was.)
    small = 2.0 ** -75 * inp["C"].double().abs().sum(-1, keepdim=True)
    tol = (ref.H16 + 2.0 ** -14) * ay + ref.H16 * ry.abs() + drift[..., None] * ay + gone[..., None] + tiny + small
    ref.close(y, ry, tol, f"rate {rate} y")
    last = torch.stack([drift[v - 1] for v in at[1:]])
    ref.close(st, rst, ref.ssd_state_tolerance(ast, 4) - 1e-30 + last[..., None, None] * ast + tiny, f"rate {rate} states")
