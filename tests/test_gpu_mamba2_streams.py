"""The operators on packed sequences in the ways programs call them: captured into a
graph and replayed on other values, on two streams at once, and with offsets that do not
fit 32 bits.  Each result is compared bit by bit with the plain call's."""
import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
H, G, DIM = 6, 2, 6 * 64 + 2 * 2 * 128


def _cu(lens):
    return torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")


def _inputs(seed, lens):
    g = ref.gen(seed)
    T = sum(lens)
    d = dict(x=ref.randn(g, T, DIM, dtype=torch.bfloat16), dt=ref.randn(g, T, H, dtype=torch.bfloat16, scale=0.1),
             dy=ref.randn(g, T, DIM, dtype=torch.bfloat16), z=ref.randn(g, T, H * 64, dtype=torch.bfloat16),
             windows=ref.randn(g, len(lens), 3, DIM, dtype=torch.bfloat16), states=ref.randn(g, len(lens), H, 64, 128))
    return {k: v.cuda() for k, v in d.items()}


def _params(seed):
    g = ref.gen(seed)
    p = dict(w=ref.randn(g, DIM, 4, scale=0.5), b=ref.randn(g, DIM, scale=0.2), A=-torch.empty(H).uniform_(1.0, 16.0, generator=g),
             dt_bias=torch.full((H,), -4.0), D=ref.randn(g, H), nw=1 + 0.1 * ref.randn(g, H * 64))
    return {k: v.cuda() for k, v in p.items()}


def _run(p, d, cu, initial, stream=None):
    """Convolution, SSD and norm of a batch of prompts, and the gradients of the first and the last."""
    import selective_state_space_38_b200 as ssm
    kw = dict(stream=stream)
    u = ssm.ssm_conv1d_fwd(d["x"], p["w"], p["b"], cu, windows=d["windows"], has_initial=initial, **kw)
    x, B, C = (v.unflatten(1, (-1, e)) for v, e in zip(u.split([H * 64, G * 128, G * 128], 1), (64, 128, 128)))
    y = ssm.ssm_ssd_varlen_fwd(x, d["dt"], p["dt_bias"], True, p["A"], B, C, p["D"], cu, states=d["states"], has_initial=initial, **kw)
    out, rstd = ssm.ssm_gated_norm_fwd(y.flatten(1), p["nw"], d["z"], groups=G, **kw)
    gn = ssm.ssm_gated_norm_bwd(y.flatten(1), p["nw"], d["z"], out, groups=G, **kw)
    gc = ssm.ssm_conv1d_bwd(d["x"], p["w"], p["b"], cu, d["dy"], **kw)
    return [u, y, out, rstd, *gn.values(), *gc.values(), d["windows"], d["states"]]


def _equal(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("lens", [[130, 1, 0, 700, 40], [3000], [600, 600]])
def test_captured_and_replayed_on_other_values(lens):
    """One graph of every operator: ranges, whole chains and the two passes of the SSD, the second kernels of the others."""
    cu, p = _cu(lens), _params(1)
    initial = torch.tensor([i % 2 == 0 for i in range(len(lens))], device="cuda")
    d = _inputs(2, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(p, {k: v.clone() for k, v in d.items()}, cu, initial)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _run(p, d, cu, initial)
    for seed in (3, 4):
        new = _inputs(seed, lens)
        for k, v in new.items():
            d[k].copy_(v)
        graph.replay()
        want = _run(p, new, cu, initial)
        torch.cuda.synchronize()
        _equal(got, want)


def test_two_streams_at_once():
    """Calls that share the SMs: prompts on two streams, a hand-off of states in each, results as by themselves."""
    p = _params(5)
    batches = [[900, 333, 128, 70] * 3, [2000, 10] * 4]
    cus = [_cu(b) for b in batches]
    initial = [torch.ones(len(b), dtype=torch.bool, device="cuda") for b in batches]
    ins = [[_inputs(10 + 2 * k + i, b) for k in range(6)] for i, b in enumerate(batches)]
    want = [[_run(p, {n: v.clone() for n, v in d.items()}, cus[i], initial[i]) for d in ins[i]] for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(6):
        for i in range(2):
            got[i].append(_run(p, ins[i][k], cus[i], initial[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            _equal(a, b)


def test_rows_and_slots_beyond_32_bits():
    """Rows 2^20 elements apart reach past 2^31 elements; so do the states of a cache of 45000 rows."""
    import selective_state_space_38_b200 as ssm
    lens, stride = [1500, 600], 1 << 20
    T = sum(lens)
    d, p, cu = _inputs(20, lens), _params(21), _cu(lens)
    buf = torch.empty(T, stride, dtype=torch.bfloat16, device="cuda")
    wide = buf[:, 4096:4096 + DIM]
    wide.copy_(d["x"])
    out = buf[:, 8192:8192 + DIM]
    _equal([ssm.ssm_conv1d_fwd(wide, p["w"], p["b"], cu, out=out)], [ssm.ssm_conv1d_fwd(d["x"], p["w"], p["b"], cu)])
    a, b = ssm.ssm_conv1d_bwd(wide, p["w"], p["b"], cu, d["dy"], dx=out), ssm.ssm_conv1d_bwd(d["x"], p["w"], p["b"], cu, d["dy"])
    _equal(a.values(), b.values())
    n = H * 64
    z, y = buf[:, 4096:4096 + n], buf[:, 16384:16384 + n]
    _equal([ssm.ssm_gated_norm_fwd(z, p["nw"], d["z"], out=y)[0]], [ssm.ssm_gated_norm_fwd(z.contiguous(), p["nw"], d["z"])[0]])
    views = lambda t: [v.unflatten(1, (-1, e)) for v, e in zip(t.split([n, G * 128, G * 128], 1), (64, 128, 128))]
    slots = torch.tensor([44999, 44000], dtype=torch.int32, device="cuda")
    cache = torch.empty(45000, H, 64, 128, device="cuda")
    small = torch.zeros(2, H, 64, 128, device="cuda")
    got = ssm.ssm_ssd_varlen_fwd(*views(wide)[:1], d["dt"], p["dt_bias"], True, p["A"], *views(wide)[1:], p["D"], cu,
                                 states=cache, slots=slots, out=y.unflatten(1, (H, 64)), check=True)
    want = ssm.ssm_ssd_varlen_fwd(*views(d["x"])[:1], d["dt"], p["dt_bias"], True, p["A"], *views(d["x"])[1:], p["D"], cu,
                                  states=small, check=True)
    _equal([got, cache[slots.long()]], [want, small])
    rows = [t[:2] for t in (d["x"], d["dt"])]
    got = ssm.ssm_ssd_step(cache, views(rows[0])[0], rows[1], p["dt_bias"], True, p["A"], *views(rows[0])[1:], p["D"], slots=slots)
    want = ssm.ssm_ssd_step(small, views(rows[0])[0], rows[1], p["dt_bias"], True, p["A"], *views(rows[0])[1:], p["D"])
    _equal([got, cache[slots.long()]], [want, small])
    windows = torch.empty(2_000_000, 3, DIM, dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([1_999_999, 1_500_000], dtype=torch.int32, device="cuda")
    near = ref.randn(ref.gen(22), 2, 3, DIM, dtype=torch.bfloat16).cuda()
    windows[far.long()] = near
    got, want = ssm.ssm_conv1d_step(windows, rows[0], p["w"], p["b"], slots=far), ssm.ssm_conv1d_step(near, rows[0], p["w"], p["b"])
    _equal([got, windows[far.long()]], [want, near])


def test_only_empty_sequences():
    """No rows in any sequence: outputs and caches stay as they were, the sums of the gradients are zeros."""
    import selective_state_space_38_b200 as ssm
    p, d = _params(30), _inputs(31, [5])
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    u, gx, y = (torch.full((5, n), 7.0, dtype=torch.bfloat16, device="cuda") for n in (DIM, DIM, H * 64))
    windows, states = torch.full((3, 3, DIM), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((3, H, 64, 128), 5.0, device="cuda")
    x, B, C = (v.unflatten(1, (-1, e)) for v, e in zip(d["x"].split([H * 64, G * 128, G * 128], 1), (64, 128, 128)))
    ssm.ssm_conv1d_fwd(d["x"], p["w"], p["b"], cu, windows=windows, out=u)
    ssm.ssm_ssd_varlen_fwd(x, d["dt"], p["dt_bias"], True, p["A"], B, C, p["D"], cu, states=states, out=y.unflatten(1, (H, 64)), check=True)
    g = ssm.ssm_conv1d_bwd(d["x"], p["w"], p["b"], cu, d["dy"], dx=gx)
    assert all((t == 7.0).all() for t in (u, gx, y)) and (windows == 5.0).all() and (states == 5.0).all()
    assert not g["dw"].any() and not g["dbias"].any()


def test_thousands_of_short_sequences():
    """2500 sequences of no to three tokens: as in three calls of fewer."""
    import selective_state_space_38_b200 as ssm
    g = ref.gen(32)
    lens = [int(v) for v in torch.randint(0, 4, (2500,), generator=g)]
    p, d = _params(33), _inputs(34, [sum(lens)])
    states, windows = torch.randn(2500, H, 64, 128, generator=g).cuda(), ref.randn(g, 2500, 3, DIM, dtype=torch.bfloat16).cuda()

    def run(n0, n1):
        a, b = sum(lens[:n0]), sum(lens[:n1])
        s, w, cu = states[n0:n1].clone(), windows[n0:n1].clone(), _cu(lens[n0:n1])
        initial = torch.ones(n1 - n0, dtype=torch.bool, device="cuda")
        u = ssm.ssm_conv1d_fwd(d["x"][a:b], p["w"], p["b"], cu, windows=w, has_initial=initial)
        x, B, C = (v.unflatten(1, (-1, e)) for v, e in zip(u.split([H * 64, G * 128, G * 128], 1), (64, 128, 128)))
        y = ssm.ssm_ssd_varlen_fwd(x, d["dt"][a:b], p["dt_bias"], True, p["A"], B, C, p["D"], cu, states=s, has_initial=initial, check=True)
        gx = ssm.ssm_conv1d_bwd(d["x"][a:b], p["w"], p["b"], cu, d["dy"][a:b])["dx"]
        return u, y, gx, s, w

    _equal(run(0, 2500), [torch.cat(v) for v in zip(run(0, 1000), run(1000, 2000), run(2000, 2500))])
