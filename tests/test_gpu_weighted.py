"""GPU: the weighted combine and its backward (moe_combine_weighted, moe_combine_weighted_bwd)
against 64-bit references: repeated ids, empty slots with NaN weights, tokens without a row, pad and
sentinel rows, both walks of the backward, gradients against differences, streams and graphs.

Bounds (u = 2^-24): the forward rounds the first product and every fma once, so a token of n rows is
within n u sum |w y| of the exact sum, plus half a bf16 step (2^-8) for bf16 outputs.  The grad rows
are one fp32 product rounded to bf16, compared bit for bit.  dw is an exact sum rounded in fp64 and
once to fp32: within u |dw| plus H 2^-52 sum |g y|."""
import pytest
import torch

import expert_ref as ref
from combine_topk_idx_multihot_amd import binding as B
from combine_topk_idx_multihot_amd import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.moe_device_check(0)
    yield


class Case:
    def __init__(self, T, E, k, H, lb=0, EL=None, P=1, sync_free=False, extra=0, empty=0.1,
                 dup=False, workspace=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        idx = (torch.randint(0, E, (T, k), generator=g) if dup else
               torch.rand((T, E), generator=g).topk(k, 1).indices).to(torch.int32)
        idx[torch.rand((T, k), generator=g) < empty] = -1
        EL = E if EL is None else EL
        d = B.make_desc(T, k, E, lb, EL, P)
        if sync_free:
            d = B.make_desc(T, k, E, lb, EL, P, B.MOE_SYNC_FREE, False,
                            B.moe_capacity_min(d) + extra)
        self.d, self.H = d, H
        self.h, _ = B.route(d, idx.cuda())
        if not workspace:  # the walks over tokens
            h = self.h
            self.h = B.Handle(d, h.routing_map, h.tokens_per_expert, h.padded_offsets,
                              h.row_of_slot, h.status, h.host_status, None)
        self.R = B.rows_for(d, self.h)
        self.ros = ros = self.h.row_of_slot.cpu().long()
        # weights of slots without a row are NaN: they may not reach any result
        w = torch.randn((T, k), generator=g)
        self.w = torch.where(ros >= 0, w, torch.full_like(w, float("nan")))
        self.Y = torch.randn((self.R, H), generator=g).to(torch.bfloat16)
        hole = torch.ones(self.R, dtype=torch.bool)
        hole[ros[ros >= 0]] = False
        self.Y[hole] = float("nan")  # pad and sentinel rows too
        self.g = torch.randn((T, H), generator=g).to(torch.bfloat16)
        # the first slot of every row and its weight with its repeats', added in slot order
        self.first = torch.zeros((T, k), dtype=torch.bool)
        self.W = torch.zeros((T, k))
        for j in range(k):
            same = (ros[:, :j] == ros[:, j:j + 1]).any(1) if j else torch.zeros(T, dtype=torch.bool)
            self.first[:, j] = (ros[:, j] >= 0) & ~same
            W = self.w[:, j].clone()
            for q in range(j + 1, k):
                W = torch.where(ros[:, q] == ros[:, j], W + self.w[:, q], W)
            self.W[:, j] = W

    def gpu(self):
        return self.Y.cuda(), self.w.cuda(), self.g.cuda()

    def forward(self):
        """fp64 out and its bound."""
        rows = self.Y[self.ros.clamp_min(0)].double() if self.R else torch.zeros((*self.ros.shape, self.H)).double()
        terms = torch.where(self.first[:, :, None], rows * self.W[:, :, None].double(),
                            torch.zeros((), dtype=torch.float64))
        n = self.first.sum(1)[:, None]
        return terms.sum(1), n * ref.U * terms.abs().sum(1) * (1 + 1e-6)

    def backward(self):
        """bf16 grad rows (exact) and fp64 dw with its bound."""
        gr = torch.zeros((self.R, self.H), dtype=torch.bfloat16)
        t, j = self.first.nonzero(as_tuple=True)
        gr[self.ros[t, j]] = (self.g[t].float() * self.W[t, j][:, None]).to(torch.bfloat16)
        rows = self.Y[self.ros.clamp_min(0)].double() if self.R else torch.zeros((*self.ros.shape, self.H)).double()
        prod = torch.where((self.ros >= 0)[:, :, None], rows * self.g[:, None].double(),
                           torch.zeros((), dtype=torch.float64))
        dw = prod.sum(2)
        return gr, dw, ref.U * dw.abs() + self.H * 2.0 ** -52 * prod.abs().sum(2)


def bits(t):
    return t.cpu().view(torch.int16)


CASES = {
    "list": dict(T=640, E=24, k=4, H=512, lb=4, EL=16, P=4),
    "list_all_local": dict(T=1100, E=16, k=8, H=2048, P=16),
    "tokens": dict(T=640, E=24, k=4, H=512, lb=4, EL=16, P=4, workspace=False),
    "tokens_wide": dict(T=130, E=8, k=2, H=4096, workspace=False),
    "tokens_odd_h": dict(T=77, E=8, k=3, H=768, P=3, workspace=False),
    "share": dict(T=900, E=64, k=4, H=1280, lb=60, EL=4, sync_free=True, extra=9),
    "sync_free_list": dict(T=700, E=16, k=8, H=256, P=8, sync_free=True),
    "dups": dict(T=500, E=5, k=7, H=256, dup=True, P=2),
    "dups_tokens": dict(T=500, E=5, k=7, H=512, dup=True, workspace=False),
    "one_token": dict(T=1, E=128, k=8, H=2048, sync_free=True, empty=0.0),
    "k1": dict(T=33, E=4, k=1, H=256),
    "k64": dict(T=20, E=80, k=64, H=256, empty=0.5),
    "all_empty": dict(T=40, E=8, k=4, H=256, empty=1.1),
    "all_empty_sync_free": dict(T=600, E=8, k=4, H=256, empty=1.1, sync_free=True),
}


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    c = Case(seed=len(name), **CASES[name])
    Y, w, _ = c.gpu()
    want, bound = c.forward()
    out = torch.full((c.d.T, c.H), 9.0, device="cuda")
    B.moe_combine_weighted(c.d, c.h, Y, c.H, c.R, w, out)
    ref.check_close(out.cpu(), want, bound, name)
    b = B.combine_weighted(c.d, c.h, Y, w)
    assert torch.equal(b, out.to(torch.bfloat16))
    alone = c.first.sum(1) == 0
    assert (bits(b)[alone] == 0).all()  # +0 without a row


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    c = Case(seed=len(name), **CASES[name])
    Y, w, g = c.gpu()
    gr = torch.full((c.R, c.H), 9.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((c.d.T, c.d.k), 9.0, device="cuda")
    B.moe_combine_weighted_bwd(c.d, c.h, g, Y, c.H, c.R, w, gr, dw)
    want, wdw, bound = c.backward()
    assert torch.equal(bits(gr), bits(want)), name
    ref.check_close(dw.cpu(), wdw, bound, name)


def test_unit_weights_give_the_plain_combine():
    c = Case(600, 12, 4, 768, P=2)
    Y, w, g = c.gpu()
    one = torch.ones_like(w)
    assert torch.equal(bits(B.combine_weighted(c.d, c.h, Y, one)), bits(B.combine(c.d, c.h, Y)))
    a, b = B.combine_weighted_bwd(c.d, c.h, g, Y, one), B.combine_bwd(c.d, c.h, g, c.R, Y)
    assert torch.equal(bits(a[0]), bits(b[0])) and torch.equal(a[1], b[1])


def test_infinite_values_stay_in_their_token():
    c = Case(50, 8, 2, 256, empty=0.0)
    Y, w, _ = c.gpu()
    clean = B.combine_weighted(c.d, c.h, Y, w)
    Y[c.ros[7, 1]] = float("inf")
    w[9, 0] = float("nan")
    out = B.combine_weighted(c.d, c.h, Y, w)
    keep = [t for t in range(50) if t not in (7, 9)]
    assert torch.equal(out[keep], clean[keep])
    assert torch.isinf(out[7]).all() and torch.isnan(out[9]).all()


def layer(c, Y, w):
    h = c.h
    return ops.combine_weighted(Y, w, h.routing_map, h.tokens_per_expert, h.padded_offsets,
                                h.row_of_slot, h.status, h.workspace, c.d.E, c.d.local_begin,
                                c.d.pad_multiple, c.d.capacity)


@pytest.mark.parametrize("sync_free", [False, True])
def test_autograd(sync_free):
    c = Case(300, 16, 4, 512, lb=3, EL=11, P=4, sync_free=sync_free)
    Y, w, g = c.gpu()
    Y.requires_grad_(True), w.requires_grad_(True)
    out = layer(c, Y, w)
    gy, gw = torch.autograd.grad(out, (Y, w), g)
    want, wdw, bound = c.backward()
    assert torch.equal(bits(gy), bits(want))
    ref.check_close(gw.cpu(), wdw, bound, "dw")


def test_gradients_against_differences():
    """The sum is linear in the weights and in the rows, so a central difference of any step has no
    truncation error: only the forward's rounding, n u sum |w y| per output on either side."""
    c = Case(120, 10, 3, 256, dup=True)
    Y, w, g = c.gpu()
    G = g.float()
    ok = c.ros.cuda() >= 0
    rng = torch.Generator(device="cuda").manual_seed(2)
    v = torch.where(ok, torch.randn(w.shape, generator=rng, device="cuda"), torch.zeros_like(w))

    def loss(Yv, wv):
        out = torch.empty((c.d.T, c.H), device="cuda")
        B.moe_combine_weighted(c.d, c.h, Yv, c.H, c.R, wv, out)
        return (out.double() * G.double()).sum()

    gr, dw = B.combine_weighted_bwd(c.d, c.h, g, Y, w)
    data = torch.zeros(c.R, 1, dtype=torch.bool, device="cuda")
    data[c.ros[c.ros >= 0].cuda()] = True
    mag = torch.where(data, Y.double().abs(), torch.zeros((), dtype=torch.float64, device="cuda"))
    ros = c.ros.cuda().clamp_min(0)
    size = ((mag[ros] * ok[:, :, None]) * G.double().abs()[:, None]).sum(2)  # sum |g y| per slot
    rng_w = torch.where(ok, w.abs() + v.abs(), torch.zeros_like(w)).double()
    # every forward value: k products or fmas, and w +- v (and merging repeats) rounded once each
    slack = float((2 * c.d.k + 2) * ref.U * c.d.k * (rng_w * size).sum())
    got = (loss(Y, w + v) - loss(Y, w - v)) / 2
    assert abs(float(got - (dw.double() * v.double()).sum())) <= slack
    # rows: Y +- D exactly representable (one unit in the last bf16 place of 2^k steps: D = Y / 2)
    D = torch.where(data, Y.float(), torch.zeros((), device="cuda")) * 0.5
    Yp, Ym = (Y.float() + D).to(torch.bfloat16), (Y.float() - D).to(torch.bfloat16)
    step = torch.where(data, (Yp.double() - Ym.double()) / 2, torch.zeros((), dtype=torch.float64, device="cuda"))
    got = (loss(Yp, w) - loss(Ym, w)) / 2
    W = torch.where(ok, w.abs(), torch.zeros_like(w)).double()
    # the grad rows are bf16 (half a step 2^-8 each), the forward fp32
    slack = float((2.0 ** -8 + (2 * c.d.k + 2) * ref.U * c.d.k) * 2 * (W * size).sum())
    assert abs(float(got - (gr.double() * step).sum())) <= slack


@pytest.mark.parametrize("sync_free", [False, True])
def test_row_gradients_against_differences_token_by_token(sync_free):
    """As above for the rows, along a step whose sign is the gradient's, so that no two terms of a token
    cancel: D = |Y| / 2 * sign(W g).  Per token, with S = sum |W g step| (the difference itself), the
    grad rows' rounding to bf16 is within 2^-8 S, and the forward's, at most k roundings of every output
    at either end, within k u sum |W g| (|Y + D| + |Y - D|) / 2.  The forward and the gradient use the same
    fp32 W.  A gradient that is zero, negated, without its weight or zero in one row of each token is outside."""
    c = Case(120, 10, 3, 256, dup=True, sync_free=sync_free)
    Y, w, g = c.gpu()
    G = g.double()
    gr = B.combine_weighted_bwd(c.d, c.h, g, Y, w)[0].double()
    # every data row's token and merged weight
    t, j = (i.cuda() for i in c.first.nonzero(as_tuple=True))
    r, W = c.ros.cuda()[t, j], c.W.cuda()[t, j].double()[:, None]
    grad = W * G[t]
    D = Y[r].double().abs() / 2 * torch.sign(grad)
    ends = []
    for side in (1, -1):
        Ys = Y.clone()
        Ys[r] = (Y[r].double() + side * D).to(torch.bfloat16)
        out = torch.empty((c.d.T, c.H), device="cuda")
        B.moe_combine_weighted(c.d, c.h, Ys, c.H, c.R, w, out)
        ends.append((Ys[r].double(), (out.double() * G).sum(1)))
    (yp, lp), (ym, lm) = ends
    step, got = (yp - ym) / 2, (lp - lm) / 2

    def per_token(rows):
        return torch.zeros(c.d.T, dtype=torch.float64, device="cuda").index_add_(0, t, rows.sum(1))

    slack = per_token(2.0 ** -8 * (grad * step).abs()
                      + c.d.k * ref.U * grad.abs() * (yp.abs() + ym.abs()) / 2 * (1 + 1e-6))

    def off(rows):
        return (got - per_token(rows * step)).abs() > slack

    assert not off(gr[r]).any()
    some = per_token(grad.abs()) > 0
    assert int(some.sum()) > 100
    for wrong in (torch.zeros_like(grad), -gr[r]):
        assert off(wrong)[some].all()
    one = gr[r].clone()
    first = c.first.cumsum(1)[c.first].cuda() == 1  # the first row of every token
    one[first] = 0
    # leaving that row out takes at least (1 - 2^-8) of its share away: outside the slack where that is
    # more than twice the slack (a row whose weight is next to nothing is not)
    share = per_token(first[:, None] * (grad * step).abs()) * (1 - 2.0 ** -8) > 2 * slack
    assert int(share.sum()) > 100 and off(one)[share].all()
    far = per_token(((W - 1).abs() > 0.1) * grad.abs()) == per_token(grad.abs())  # no weight near 1
    assert int((far & some).sum()) > 80 and off(G[t])[far & some].all()


def test_prepared_and_streams():
    c = Case(400, 16, 4, 512, P=4)
    Y, w, g = c.gpu()
    out, want = torch.zeros((400, 512), device="cuda"), torch.empty((400, 512), device="cuda")
    B.moe_combine_weighted(c.d, c.h, Y, 512, c.R, w, want)
    gr, dw = B.combine_weighted_bwd(c.d, c.h, g, Y, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gr2, dw2 = torch.zeros_like(gr), torch.zeros_like(dw)
    torch.cuda.synchronize()
    B.PreparedCombineWeighted(c.d, c.h, Y, 512, w, out, stream=s)(c.R)
    B.PreparedCombineWeightedBwd(c.d, c.h, g, Y, 512, w, gr2, dw2, stream=s)(c.R)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(gr, gr2) and torch.equal(dw, dw2)


def test_graph_replays():
    """Forward and backward captured, replayed on new values with eager calls in between."""
    c = Case(200, 16, 4, 512, sync_free=True)
    Y, w, g = c.gpu()

    def run():
        return (B.combine_weighted(c.d, c.h, Y, w), *B.combine_weighted_bwd(c.d, c.h, g, Y, w))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in range(4):
        rng = torch.Generator(device="cuda").manual_seed(seed)
        for t in (Y, w, g):
            t.copy_(torch.randn(t.shape, generator=rng, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, run())), seed


def test_backward_captured():
    """The op's forward and backward captured together, the gradients taken with autograd.grad."""
    c = Case(200, 16, 4, 512, sync_free=True, empty=0.0)
    Y, w, g = c.gpu()
    Y = torch.nan_to_num(Y).requires_grad_(True)
    w.requires_grad_(True)

    def step():
        return torch.autograd.grad(layer(c, Y, w), (Y, w), g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        with torch.no_grad():
            w.copy_(torch.randn(w.shape, device="cuda",
                                generator=torch.Generator(device="cuda").manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(kept, step())), seed


def test_op_check():
    c = Case(30, 8, 2, 256)
    Y, w, _ = c.gpu()
    Y = torch.nan_to_num(Y)
    h = c.h
    args = (Y.requires_grad_(True), torch.nan_to_num(w).requires_grad_(True), h.routing_map,
            h.tokens_per_expert, h.padded_offsets, h.row_of_slot, h.status, h.workspace, 8, 0, 1, 0)
    torch.library.opcheck(ops.combine_weighted, args,
                          test_utils=("test_schema", "test_faketensor", "test_autograd_registration"))
