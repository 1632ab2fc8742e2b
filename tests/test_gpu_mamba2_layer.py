"""The operators together, as a Mamba-2 layer uses them: prompts of different
lengths through convolution, SSD and gated norm, then tokens one at a time from the
caches, against one longer pass; and the gradients of convolution and norm chained
around a plain SSD."""
import pytest
import torch

import mamba2_ref as ref

pytestmark = pytest.mark.gpu
H, G = 4, 2
DIN, DIM = H * 64, H * 64 + 2 * G * 128
F64 = torch.float64


class Layer:
    """Parameters of one layer and its caches; `rows` are the projection's [z | x B C | dt]."""

    def __init__(self, seed, slots):
        g = ref.gen(seed)
        self.p = dict(w=ref.randn(g, DIM, 4, scale=0.5), b=ref.randn(g, DIM, scale=0.2), A=-torch.empty(H).uniform_(1.0, 16.0, generator=g),
                      dt_bias=torch.full((H,), -4.0) + ref.randn(g, H, scale=0.5), D=ref.randn(g, H), nw=1 + 0.1 * ref.randn(g, DIN))
        self.d = {k: v.cuda() for k, v in self.p.items()}
        self.windows = torch.zeros(slots, 3, DIM, dtype=torch.bfloat16, device="cuda")
        self.states = torch.zeros(slots, H, 64, 128, device="cuda")

    def split(self, rows):
        z, xbc, dt = rows[:, :DIN], rows[:, DIN:DIN + DIM], rows[:, DIN + DIM:]
        return z, xbc, dt

    def heads(self, y):
        return (y[:, :DIN].unflatten(1, (H, 64)), y[:, DIN:DIN + G * 128].unflatten(1, (G, 128)), y[:, DIN + G * 128:].unflatten(1, (G, 128)))

    def prompts(self, rows, cu, slots, has_initial):
        import selective_state_space_38_b200 as ssm
        z, xbc, dt = self.split(rows)
        d = self.d
        x, B, C = self.heads(ssm.ssm_conv1d_fwd(xbc, d["w"], d["b"], cu, windows=self.windows, slots=slots, has_initial=has_initial))
        y = ssm.ssm_ssd_varlen_fwd(x, dt, d["dt_bias"], True, d["A"], B, C, d["D"], cu, states=self.states, slots=slots,
                                   has_initial=has_initial, check=True)
        return ssm.ssm_gated_norm_fwd(y.flatten(1), d["nw"], z, groups=G)[0]

    def tokens(self, rows, slots):
        import selective_state_space_38_b200 as ssm
        z, xbc, dt = self.split(rows)
        d = self.d
        x, B, C = self.heads(ssm.ssm_conv1d_step(self.windows, xbc, d["w"], d["b"], slots=slots))
        y = ssm.ssm_ssd_step(self.states, x, dt, d["dt_bias"], True, d["A"], B, C, d["D"], slots=slots)
        return ssm.ssm_gated_norm_fwd(y.flatten(1), d["nw"], z, groups=G)[0]

    def exact(self, rows, lens):
        """The layer in float64 with the stored roundings of its intermediate rows to bfloat16 left out."""
        z, xbc, dt = (v.double() for v in self.split(rows))
        y, _, _ = ref.conv(xbc, self.p["w"], self.p["b"], lens)
        x, B, C = self.heads(y)
        out, _ = ref.ssd(dict(x=x, dt=dt, dt_bias=self.p["dt_bias"], A=self.p["A"], B=B, C=C, D=self.p["D"]), lens)
        return ref.norm(out.flatten(1), self.p["nw"].double(), z, G, 1e-5, True)[0]


def _cu(lens):
    return torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")


def test_prompts_then_tokens_equal_one_longer_pass():
    lens, more = [37, 1, 140], 5
    layer = Layer(1, 5)
    full = [ref.randn(ref.gen(10 + i), n + more, DIN + DIM + H, dtype=torch.bfloat16) for i, n in enumerate(lens)]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    got = [[] for _ in lens]
    out = layer.prompts(torch.cat([f[:n] for f, n in zip(full, lens)]).cuda(), _cu(lens), slots, None)
    for i, (a, b) in enumerate(zip(ref.offsets(lens), ref.offsets(lens)[1:])):
        got[i].append(out[a:b])
    # two more tokens each as a packed pass that goes on from the caches, the others one at a time
    two = torch.cat([f[n:n + 2] for f, n in zip(full, lens)]).cuda()
    out = layer.prompts(two, _cu([2, 2, 2]), slots, torch.ones(3, dtype=torch.bool, device="cuda"))
    for i in range(3):
        got[i].append(out[2 * i:2 * i + 2])
    for t in range(2, more):
        out = layer.tokens(torch.stack([f[n + t] for f, n in zip(full, lens)]).cuda(), slots)
        for i in range(3):
            got[i].append(out[i:i + 1])
    other = Layer(1, 5)
    longer = [n + more for n in lens]
    whole = other.prompts(torch.cat(full).cuda(), _cu(longer), slots, None)
    exact = layer.exact(torch.cat(full), longer)
    for i, (a, b) in enumerate(zip(ref.offsets(longer), ref.offsets(longer)[1:])):
        pieces = torch.cat(got[i])
        # three rows of bfloat16 on the way (the convolution's, the SSD's with its two operand
        # roundings, the norm's), each off by at most 2^-8 of its values, which the norm's
        # division may add up: 2-norms within six of them
        for v in (pieces, whole[a:b]):
            e = (v.cpu().double() - exact[a:b]).norm() / exact[a:b].norm()
            assert e <= 6 * ref.H16, (i, float(e))
    assert torch.equal(layer.windows, other.windows)
    # float32 states of the same inputs by two routes, the step's and the chunks'
    e = (layer.states - other.states).norm() / other.states.norm()
    assert e <= 2e-6, float(e)


def test_captured_decode_with_padding():
    """A captured decode step on a padded batch, replayed as rows come and go."""
    layer, eager = Layer(2, 4), Layer(2, 4)
    rows = torch.zeros(4, DIN + DIM + H, dtype=torch.bfloat16, device="cuda")
    slots = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.tokens(rows, slots)  # every row padding: nothing is written
    torch.cuda.current_stream().wait_stream(side)
    assert (layer.states == 0).all() and (layer.windows == 0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.tokens(rows, slots)
    for i, live in enumerate([[0, 1], [0, 1, 2, 3], [2], [3, 0]]):
        new = ref.randn(ref.gen(20 + i), 4, DIN + DIM + H, dtype=torch.bfloat16).cuda()
        where = torch.tensor(live + [-1] * (4 - len(live)), dtype=torch.int32, device="cuda")
        rows.copy_(new), slots.copy_(where)
        graph.replay()
        want = eager.tokens(new, where)
        torch.cuda.synchronize()
        n = len(live)
        assert torch.equal(out[:n], want[:n])
        assert torch.equal(layer.states, eager.states) and torch.equal(layer.windows, eager.windows)


def test_gradients_chain():
    """loss = sum(weights x norm(silu(conv(x)) gated by z)): the norm's gradient through the convolution's."""
    import selective_state_space_38_b200 as ssm
    lens, dim = [70, 33], 128
    g = ref.gen(3)
    x, z, up = (ref.randn(g, sum(lens), dim) for _ in range(3))
    w, b, nw = ref.randn(g, dim, 4, scale=0.5), ref.randn(g, dim, scale=0.2), 1 + 0.1 * ref.randn(g, dim)
    c = [v.cuda() for v in (x, z, up, w, b, nw)]
    cu = _cu(lens)
    y = ssm.ssm_conv1d_fwd(c[0], c[3], c[4], cu)
    gn = ssm.ssm_gated_norm_bwd(y, c[5], c[1], c[2], groups=2)
    gc = ssm.ssm_conv1d_bwd(c[0], c[3], c[4], cu, gn["dx"])
    leaves = [v.double().requires_grad_() for v in (x, z, w, b, nw)]
    parts, at = [], ref.offsets(lens)
    for i in range(2):
        parts.append(ref.conv_sequence(leaves[0][at[i]:at[i + 1]], leaves[2], leaves[3], torch.zeros(3, dim, dtype=F64))[0])
    out, _ = ref.norm(torch.cat(parts), leaves[4], leaves[1], 2, 1e-5, True)
    want = torch.autograd.grad(out, leaves, up.double())
    for got, exact, name in zip((gc["dx"], gn["dz"], gc["dw"], gc["dbias"], gn["dweight"]), want, ("dx", "dz", "dw", "dbias", "dweight")):
        e = (got.cpu().double() - exact).norm() / exact.norm()
        assert e <= 2.0 ** -17, (name, float(e))  # some ten float32 operations of 2^-21 or finer in a row
