"""GPU parity of the packed SSD (ssm_ssd_varlen_fwd) and its decode step
(ssm_ssd_step) against the float64 recurrence on the same stored inputs."""
import ctypes

import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu


def _dev(inp):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in inp.items()}


def _cu(lens):
    return torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")


def _call(inp, lens, states=None, slots=None, initial=None, out=None, **kw):
    import selective_state_space_38_b200 as ssm
    d = _dev(inp)
    y = ssm.ssm_ssd_varlen_fwd(d["x"], d["dt"], d.get("dt_bias"), inp.get("softplus", True), d["A"], d["B"], d["C"],
                               d.get("D"), _cu(lens), states=states, slots=slots, has_initial=initial, out=out,
                               check=True, **kw)
    torch.cuda.synchronize()
    return y


def _check(inp, lens, pad=0, with_states=True, initial=None, seed=0, what=""):
    g = ref.gen(1000 + seed)
    H, G = inp["x"].shape[1], inp["B"].shape[1]
    n = len(lens)
    states = ref.randn(g, n + 2, H, 64, 128) if with_states else None
    slots = torch.randperm(n + 2, generator=g)[:n].to(torch.int32) if with_states else None
    out = torch.full(tuple(inp["x"].shape), 7.0, dtype=torch.bfloat16, device="cuda")
    st = states.cuda() if with_states else None
    y = _call(inp, lens, st, None if slots is None else slots.cuda(),
              None if initial is None else torch.tensor(initial, device="cuda"), out=out)
    ry, rst = ref.ssd(inp, lens, states, slots, initial)
    ay, ast = ref.ssd(inp, lens, states, slots, initial, absolute=True)
    T = sum(lens)
    assert (y[T:].cpu() == 7.0).all(), "rows behind the last sequence"
    ref.close(y[:T], ry[:T], ref.ssd_y_tolerance(ry[:T], ay[:T]), f"{what} y")
    e = (y[:T].cpu().double() - ry[:T]).norm() / ry[:T].norm()
    assert e <= 5e-3, f"{what}: 2-norm of the error {e:.2e}"
    if with_states:
        chunks = max(lens) // 128 + 2
        untouched = [s for s in range(n + 2) if s not in [int(v) for v, ln in zip(slots, lens) if ln]]
        assert torch.equal(st.cpu()[untouched], states[untouched]), "cache rows of no sequence"
        used = [int(v) for v, ln in zip(slots, lens) if ln]
        ref.close(st[used], rst[used], ref.ssd_state_tolerance(ast[used], chunks), f"{what} states")
        e = (st[used].cpu().double() - rst[used]).norm() / rst[used].norm()
        assert e <= 2e-6, f"{what}: 2-norm of the states' error {e:.2e}"


@pytest.mark.parametrize("L", [1, 2, 127, 128, 129, 300])
def test_one_sequence(L):
    inp = ref.ssd_inputs(ref.gen(L), L, 2, 1)
    _check(inp, [L], what=f"L={L}")


@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (6, 2), (4, 4), (5, 1)])
def test_head_layouts(H, G):
    """Odd heads per group leave the second head of the last pair absent."""
    lens = [130, 5]
    _check(ref.ssd_inputs(ref.gen(H * 10 + G), sum(lens), H, G), lens, initial=[True, False], seed=H, what=f"H={H} G={G}")


def test_packed_lengths_slots_and_rows_behind():
    lens = [1, 0, 200, 128, 3, 0, 65, 257]
    inp = ref.ssd_inputs(ref.gen(5), sum(lens) + 9, 4, 2)
    _check(inp, lens, pad=9, initial=[True, True, False, True, True, False, False, True], what="packed")


def test_no_states():
    lens = [140, 30]
    _check(ref.ssd_inputs(ref.gen(6), sum(lens), 2, 1), lens, with_states=False, what="no states")


@pytest.mark.parametrize("L", [1024, 1025, 2500])
def test_segments_hand_the_state_on(L):
    lens = [3, L, 40]
    inp = ref.ssd_inputs(ref.gen(L), sum(lens), 2, 1)
    _check(inp, lens, initial=[False, True, False], what=f"segments L={L}")


@pytest.mark.parametrize("H,lens", [(100, [256, 256, 256]), (61, [300, 1, 0, 129, 512, 40]), (8, [128] * 45)])
def test_ranges_hand_the_state_on(H, lens):
    """More chains than SMs: a CTA's range begins and ends inside chains."""
    inp = ref.ssd_inputs(ref.gen(H), sum(lens), H, 1)
    _check(inp, lens, initial=[i % 2 == 0 for i in range(len(lens))], what=f"ranges H={H}")


@pytest.mark.parametrize("dt_range", [(1e-5, 1e-4), (0.5, 2.0), (5.0, 20.0)])
def test_decay_ranges(dt_range):
    """From no decay within a chunk to a chunk of one step (|dt A| above 110)."""
    lens = [200, 77]
    inp = ref.ssd_inputs(ref.gen(11), sum(lens), 4, 1, dt_range=dt_range)
    inp["A"] = torch.tensor([-16.0, -1.0, -9.0, -0.01])
    _check(inp, lens, initial=[True, False], what=f"dt {dt_range}")


@pytest.mark.parametrize("rate", [0.3, 0.62, 0.7, 1.0, 1.3, 3.0])
def test_equal_decay_of_both_heads(rate):
    """Both heads of a pair decay by about `rate` a step: the widest spans of the factors within a chunk."""
    lens = [260]
    inp = ref.ssd_inputs(ref.gen(21), 260, 2, 1)
    inp["dt"].zero_()
    inp["dt_bias"] = torch.full((2,), float(torch.log(torch.expm1(torch.tensor(0.1)))))
    inp["A"] = torch.tensor([-10.0 * rate, -9.9 * rate])
    inp["D"] = None
    _check(inp, lens, initial=[True], what=f"rate {rate}")


@pytest.mark.parametrize("rates", [(0.01, 1.0), (1.0, 0.01), (1.0, 4.0), (4.0, 0.01), (2.4, 2.6)])
def test_decays_of_a_pair_of_different_kinds(rates):
    """The two heads of a pair decay by these rates a step: 128 steps of 0.01 span little, of 1 too much for factors of
    the columns alone, of 4 too much for factors of 16 columns; 16 of 2.4 and 2.6 lie about their limit.  The second
    sequence's steps vary fourfold, and some are next to nothing."""
    lens = [260, 140]
    inp = ref.ssd_inputs(ref.gen(22), sum(lens), 2, 1)
    steps = torch.full((sum(lens), 2), 0.1)
    steps[260:] = 0.05 + 0.15 * torch.rand(140, 2, generator=ref.gen(23))
    steps[270:275] = 1e-6
    inp["dt"] = torch.log(torch.expm1(steps)).to(torch.bfloat16)
    inp["dt_bias"] = None
    inp["A"] = torch.tensor([-10.0 * r for r in rates])
    inp["D"] = None
    _check(inp, lens, initial=[True, True], what=f"rates {rates}")


def test_without_bias_skip_and_softplus():
    lens = [150]
    inp = ref.ssd_inputs(ref.gen(12), 150, 2, 1)
    inp["dt"] = (inp["dt"].float().abs() * 0.3).to(torch.bfloat16)
    inp["D"] = None
    bias = inp.pop("dt_bias")
    inp["softplus"] = False
    y = _call(inp, lens)
    ry, _ = ref.ssd(inp, lens)
    inp2 = dict(inp, x=inp["x"].abs(), B=inp["B"].abs(), C=inp["C"].abs())
    ay, _ = ref.ssd(inp2, lens)
    ref.close(y, ry, ref.ssd_y_tolerance(ry, ay), "softplus off")
    assert bias is not None


def test_slices_of_wider_rows():
    """x, B and C as slices of the convolution's rows, dt of the projection's, out of a wider buffer."""
    H, G, T = 4, 1, 190
    inp = ref.ssd_inputs(ref.gen(13), T, H, G)
    wide = torch.full((T, H * 64 + 256 + 8), 9.0, dtype=torch.bfloat16)
    wide[:, :H * 64] = inp["x"].reshape(T, -1)
    wide[:, H * 64:H * 64 + 128] = inp["B"][:, 0]
    wide[:, H * 64 + 128:H * 64 + 256] = inp["C"][:, 0]
    proj = torch.full((T, 37), 3.0, dtype=torch.bfloat16)
    proj[:, 30:30 + H] = inp["dt"]
    wide, proj = wide.cuda(), proj.cuda()
    v = dict(inp, x=wide[:, :H * 64].unflatten(1, (H, 64)), B=wide[:, H * 64:H * 64 + 128].unflatten(1, (1, 128)),
             C=wide[:, H * 64 + 128:H * 64 + 256].unflatten(1, (1, 128)), dt=proj[:, 30:30 + H])
    buf = torch.full((T, H * 64 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    a = _call(v, [100, 90], out=buf[:, :H * 64].unflatten(1, (H, 64)))
    b = _call(inp, [100, 90])
    assert torch.equal(a, b) and (buf[:, H * 64:] == 7.0).all()


def test_other_sequences_values_do_not_matter():
    """NaN and infinities in a neighbouring sequence and behind the last one leave a sequence as it was."""
    lens = [70, 60, 50]
    inp = ref.ssd_inputs(ref.gen(14), sum(lens) + 40, 2, 1)
    a = _call(inp, lens)
    bad = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in inp.items()}
    for k in ("x", "B", "C", "dt"):
        bad[k][70:130] = float("nan")
        bad[k][180:] = float("inf")
    b = _call(bad, lens)
    assert torch.equal(a[:70], b[:70]) and torch.equal(a[130:180], b[130:180])


def test_slot_outside_the_cache_is_none():
    lens = [40, 50]
    inp = ref.ssd_inputs(ref.gen(15), 90, 2, 1)
    states = ref.randn(ref.gen(16), 3, 2, 64, 128).cuda()
    keep = states.clone()
    initial = torch.tensor([True, True], device="cuda")
    y = _call(inp, lens, states, torch.tensor([-1, 7], dtype=torch.int32, device="cuda"), initial)
    assert torch.equal(states, keep)
    assert torch.equal(y, _call(inp, lens))


def test_bad_table_is_reported_and_writes_nothing():
    import selective_state_space_38_b200 as ssm
    inp = _dev(ref.ssd_inputs(ref.gen(17), 100, 2, 1))
    states = torch.full((2, 2, 64, 128), 3.0, device="cuda")
    for table in ([0, 80, 60], [0, 50, 101], [-1, 50, 100]):
        out = torch.full((100, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ssm.SSMError) as e:
            ssm.ssm_ssd_varlen_fwd(inp["x"], inp["dt"], inp["dt_bias"], True, inp["A"], inp["B"], inp["C"], inp["D"],
                                   torch.tensor(table, dtype=torch.int32, device="cuda"), states=states, out=out, check=True)
        assert e.value.code == 1
        assert (out == 7.0).all() and (states == 3.0).all()


def test_split_calls_continue():
    """Two calls, the second from the states of the first, against one call."""
    inp = ref.ssd_inputs(ref.gen(18), 300, 2, 1)
    states = torch.zeros(1, 2, 64, 128, device="cuda")
    whole = torch.zeros(1, 2, 64, 128, device="cuda")
    y = _call(inp, [300], whole)
    first = {k: v[:150] if k in ("x", "dt", "B", "C") else v for k, v in inp.items()}
    rest = {k: v[150:] if k in ("x", "dt", "B", "C") else v for k, v in inp.items()}
    ya = _call(first, [150], states)
    yb = _call(rest, [150], states, initial=torch.tensor([True], device="cuda"))
    ry, rst = ref.ssd(inp, [300], torch.zeros(1, 2, 64, 128))
    ay, ast = ref.ssd(inp, [300], torch.zeros(1, 2, 64, 128), absolute=True)
    for v in (y, torch.cat([ya, yb])):
        ref.close(v, ry, ref.ssd_y_tolerance(ry, ay), "split y")
    for v in (whole, states):
        ref.close(v, rst, ref.ssd_state_tolerance(ast, 5), "split states")


@pytest.mark.parametrize("spin_limit", [0, 500])
def test_handoff_wait_timeout_is_reported(spin_limit):
    """A hand-off flag that nothing sets: the wait gives up, the kernel ends, the status says so, and the next
    call on the workspace is right."""
    import selective_state_space_38_b200 as ssm
    lib = ssm.get_lib()
    H, lens = 100, [256, 256, 256]  # 150 chains of two chunks on 148 SMs: ranges of three chunks split every third
    T = sum(lens)
    inp = ref.ssd_inputs(ref.gen(19), T, H, 1)
    d = _dev(inp)
    dims = ssm.SsdPackedDims(T, len(lens), 0, H, 64, 1, 128, H * 64, H, 128, 128, H * 64, ssm.SSM_BF16)
    n = ctypes.c_size_t(0)
    assert lib.ssm_ssd_varlen_fwd_workspace_size(ctypes.byref(dims), ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    out = torch.zeros(T, H, 64, dtype=torch.bfloat16, device="cuda")
    cu = _cu(lens)
    sp = torch.cuda.current_stream().cuda_stream
    args = [d["x"].data_ptr(), d["dt"].data_ptr(), d["dt_bias"].data_ptr(), 1, d["A"].data_ptr(), d["B"].data_ptr(),
            d["C"].data_ptr(), d["D"].data_ptr(), cu.data_ptr(), None, None, None, out.data_ptr(), ws.data_ptr(), n.value]
    assert lib.ssm_debug_ssd_varlen_flag_timeout(*args, spin_limit, ctypes.byref(dims), sp) == 0
    assert lib.ssm_scan_fwd_status(ws.data_ptr(), sp) == 5
    assert lib.ssm_ssd_varlen_fwd(*args, ctypes.byref(dims), sp) == 0
    assert lib.ssm_scan_fwd_status(ws.data_ptr(), sp) == 0
    assert torch.equal(out, _call(inp, lens))


def test_equal_calls_give_equal_bits_and_graph_replays():
    import selective_state_space_38_b200 as ssm
    lens = [1500, 20, 700]
    d = _dev(ref.ssd_inputs(ref.gen(20), sum(lens), 4, 1))
    cu = _cu(lens)

    def call(out=None, stream=None):
        return ssm.ssm_ssd_varlen_fwd(d["x"], d["dt"], d["dt_bias"], True, d["A"], d["B"], d["C"], d["D"], cu, out=out,
                                      stream=stream)
    a = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    out = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    for lens2 in ([1500, 20, 700], [20, 1500, 700], [0, 2220, 0], [740, 740, 740]):
        cu.copy_(_cu(lens2))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()), lens2


@pytest.mark.parametrize("H,lens", [(80, [1024] * 4), (24, [8192]), (24, [50, 1300, 128, 700] * 8)])
def test_repeated_calls_on_a_full_gpu_give_equal_bits(H, lens):
    """Every schedule with all SMs busy, eight times: what a missing wait between the warps would show."""
    import selective_state_space_38_b200 as ssm
    d = _dev(ref.ssd_inputs(ref.gen(22), sum(lens), H, 1))
    cu = _cu(lens)
    states = torch.zeros(len(lens), H, 64, 128, device="cuda")
    first = None
    for _ in range(8):
        y = ssm.ssm_ssd_varlen_fwd(d["x"], d["dt"], d["dt_bias"], True, d["A"], d["B"], d["C"], d["D"], cu, states=states, check=True)
        if first is None:
            first = (y, states.clone())
        assert torch.equal(y, first[0]) and torch.equal(states, first[1])


def _step_ref(inp, states, slots):
    x = inp["x"]
    one = dict(inp)
    ys, ya = [], []
    st, sa = states.double().clone(), states.double().abs()
    for b in range(x.shape[0]):
        row = {k: v[b:b + 1] if k in ("x", "dt", "B", "C") else v for k, v in one.items()}
        slot = torch.tensor([int(slots[b])])
        y, st = ref.ssd(row, [1], st, slot, [True])
        a, sa = ref.ssd(row, [1], sa, slot, [True], absolute=True)
        ys.append(y), ya.append(a)
    return torch.cat(ys), st, torch.cat(ya), sa


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,H,G", [(1, 1, 1), (3, 5, 1), (7, 6, 2), (2, 24, 1)])
def test_step(dtype, batch, H, G):
    import selective_state_space_38_b200 as ssm
    g = ref.gen(batch * 100 + H)
    inp = ref.ssd_inputs(g, batch, H, G, dtype=dtype)
    states = ref.randn(g, batch + 1, H, 64, 128)
    slots = torch.randperm(batch + 1, generator=g)[:batch].to(torch.int32)
    d, st = _dev(inp), states.cuda()
    y = ssm.ssm_ssd_step(st, d["x"], d["dt"], d["dt_bias"], True, d["A"], d["B"], d["C"], d["D"], slots=slots.cuda())
    ry, rst, ay, ast = _step_ref(inp, states, slots)
    # a handful of float32 steps on the state; 16 of them and the shuffles for y, and y's own rounding
    ref.close(st, rst, 2.0 ** -20 * ast + 1e-30, "step states")
    ref.close(y, ry, 2.0 ** -19 * ay + ref.half(dtype) * ry.abs() + 1e-30, "step y")


def test_step_padding_and_options():
    import selective_state_space_38_b200 as ssm
    inp = ref.ssd_inputs(ref.gen(31), 4, 2, 1)
    d = _dev(inp)
    states = ref.randn(ref.gen(32), 3, 2, 64, 128)
    st = states.cuda()
    out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([2, -1, 3, 0], dtype=torch.int32)
    ssm.ssm_ssd_step(st, d["x"], d["dt"], d["dt_bias"], True, d["A"], d["B"], d["C"], d["D"], slots=slots.cuda(), out=out)
    assert (out[1:3] == 7.0).all() and torch.equal(st[1].cpu(), states[1])
    pick = {k: v[[0, 3]] if k in ("x", "dt", "B", "C") else v for k, v in inp.items()}
    ry, rst, ay, ast = _step_ref(pick, states, torch.tensor([2, 0]))
    ref.close(out[[0, 3]], ry, 2.0 ** -19 * ay + ref.H16 * ry.abs(), "padded step y")
    ref.close(st, rst, 2.0 ** -20 * ast + 1e-30, "padded step states")


def test_step_equals_packed_rows():
    """Steps from a prompt's states go on as one longer sequence."""
    import selective_state_space_38_b200 as ssm
    inp = ref.ssd_inputs(ref.gen(33), 140, 4, 2)
    d = _dev(inp)
    st = torch.zeros(1, 4, 64, 128, device="cuda")
    first = {k: v[:130] if k in ("x", "dt", "B", "C") else v for k, v in inp.items()}
    ys = [_call(first, [130], st)]
    for t in range(130, 140):
        ys.append(ssm.ssm_ssd_step(st, d["x"][t:t + 1], d["dt"][t:t + 1], d["dt_bias"], True, d["A"], d["B"][t:t + 1],
                                   d["C"][t:t + 1], d["D"]))
    ry, rst = ref.ssd(inp, [140], torch.zeros(1, 4, 64, 128))
    ay, ast = ref.ssd(inp, [140], torch.zeros(1, 4, 64, 128), absolute=True)
    ref.close(torch.cat(ys), ry, ref.ssd_y_tolerance(ry, ay), "steps after a prompt")
    ref.close(st, rst, ref.ssd_state_tolerance(ast, 3), "states after the steps")
