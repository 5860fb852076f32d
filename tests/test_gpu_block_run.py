"""The operators between the GEMMs as they are used: one attention half of a transformer
block, forward and backward, with the FP8 linears around them,

    s, y = dropout_add_layernorm(x, residual)      end of the last branch, next norm
    q, k, v = Linear(y); q, k = rope(q, k)
    o = Linear(v)                                  (the attention core is the caller's)
    out = dropout_add(o, residual=s)

against the same run with each operator replaced by its 64-bit form on the same inputs, and
replayed from a graph.  Also: what the fused calls give is what the separate ones give."""
import numpy as np
import pytest
import torch

import rows_ref as ref
from rows_ref import close, draw, f64, vector

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, S, HQ, HK, D = 2, 72, 4, 2, 64
M, W = B * S, HQ * D


class Block:
    def __init__(self, seed, p=0.2):
        from fp8_gemms_b200 import api
        self.api, self.p = api, p
        self.x, self.res = draw((M, W), BF, seed), draw((M, W), BF, seed + 1, 2.0)
        self.w, self.b = vector(W, BF, seed + 2, 0.2, 1.0), vector(W, BF, seed + 3, 0.1)
        mats = [(HQ * D, W), (HK * D, W), (HK * D, W), (W, HK * D)]
        self.W = [draw(n, BF, seed + 4 + i, 0.05) for i, n in enumerate(mats)]
        self.lin = [api.Linear(M, k, n) for n, k in mats]
        self.dout = draw((M, W), BF, seed + 9, 1e-2)
        self.dq, self.dk = (draw((M, h * D), BF, seed + 10 + h, 1e-2).view(B, S, h, D)
                            for h in (HQ, HK))
        self.freq, self.mag = api.rope_frequencies(D, scaling=api.ROPE_BY_PARTS, factor=4.0,
                                                   context=64.0)
        self.rng = api.dropout_rng(1234, 5)

    def run(self):
        """Every tensor of the step, by name."""
        api, t = self.api, {}
        t["s"], t["y"], t["mean"], t["rstd"] = api.dropout_add_layernorm(
            self.x, self.res, self.w, self.b, self.p, self.rng, 0)
        q, k, t["v"] = (lin.forward(t["y"], Wt) for lin, Wt in zip(self.lin[:3], self.W))
        t["q0"], t["k0"] = q.view(B, S, HQ, D), k.view(B, S, HK, D)
        t["q"], t["k"] = api.rope([t["q0"], t["k0"]], self.freq, start=7, magnitude=self.mag)
        t["o"] = self.lin[3].forward(t["v"], self.W[3])
        t["out"] = api.dropout_add(t["o"], self.p, self.rng, 1, residual=t["s"])
        # backward: q's and k's gradients come from the attention core
        t["do"] = api.dropout_add_backward(self.dout, self.p, self.rng, 1)
        dv, t["dWo"] = self.lin[3].backward(t["do"])
        t["dq"], t["dk"] = api.rope_backward([self.dq, self.dk], self.freq, start=7,
                                             magnitude=self.mag)
        dys = [lin.backward(g.reshape(M, -1))[0]
               for lin, g in zip(self.lin, (t["dq"], t["dk"], dv))]
        t["dy"] = dys[0] + dys[1] + dys[2]
        t["dx"], t["dres"], t["dw"], t["db"] = api.dropout_add_layernorm_backward(
            t["dy"], self.dout, t["s"], self.w, t["mean"], t["rstd"], self.p, self.rng, 0)
        return t


def test_a_block_forward_and_backward():
    blk = Block(1)
    t = blk.run()
    torch.cuda.synchronize()
    keep, scale = ref.keep_mask(M, W, blk.p, 1234, 5)
    keep1, _ = ref.keep_mask(M, W, blk.p, 1234, 6)
    host = lambda x: x.float().cpu().numpy()
    s = torch.from_numpy(host(blk.res) + ref.dropped(host(blk.x), keep, scale)).to(BF).cuda()
    assert torch.equal(t["s"], s)
    args = (f64(s), f64(blk.w), f64(blk.b), 1e-5)
    close(f64(t["y"]), ref.norm(*args)[0], ref.norm_bounds(*args, BF)[0], "y")
    pos, f = np.broadcast_to(7 + np.arange(S), (B, S)), f64(blk.freq)
    for name, raw, inverse in [("q", t["q0"], False), ("k", t["k0"], False), ("dq", blk.dq, True),
                               ("dk", blk.dk, True)]:
        close(f64(t[name]), ref.rope(f64(raw), f, pos, False, blk.mag, inverse),
              ref.rope_bound(f64(raw), f, pos, False, blk.mag, BF, inverse), name)
    out = torch.from_numpy(host(s) + ref.dropped(host(t["o"]), keep1, scale)).to(BF).cuda()
    assert torch.equal(t["out"], out)
    do = torch.from_numpy(ref.dropped(host(blk.dout), keep1, scale)).to(BF).cuda()
    assert torch.equal(t["do"], do)
    args = (f64(t["dy"]), f64(s), f64(blk.w), f64(t["mean"]), f64(t["rstd"]))
    (dx, dw, db), (bx, bw, bb) = ref.norm_grads(*args), ref.norm_grad_bounds(*args, torch.float32, BF)
    total = dx + f64(blk.dout)
    inner = bx + 2 * ref.U * np.abs(total)
    close(f64(t["dres"]), total, inner + ref.HALF[BF] * (np.abs(total) + inner), "dres")
    inner = (inner + 2 * ref.U * np.abs(total)) * float(scale) * keep
    want = np.where(keep, total * float(scale), 0.0)
    close(f64(t["dx"]), want, inner + ref.HALF[BF] * (np.abs(want) + inner), "dx")
    close(f64(t["dw"]), dw, bw, "dweight")
    close(f64(t["db"]), db, bb, "dbias")


def test_a_block_replayed_from_a_graph():
    """Captured once: replays give the eager bits, and new masks once the offset has moved."""
    blk = Block(51)
    eager = {k: v.clone() for k, v in blk.run().items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t = blk.run()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for name, want in eager.items():
        assert torch.equal(t[name], want), name
    blk.rng[1] += 2
    g.replay()
    torch.cuda.synchronize()
    moved = {k: v.clone() for k, v in t.items()}
    for name, want in blk.run().items():
        assert torch.equal(moved[name], want), name
    assert not torch.equal(moved["s"], eager["s"])


def test_the_norm_feeds_the_cast_with_its_amax():
    """layernorm(amax_out=) then cast(amax_in=) gives the codes and scales of the cast that
    reduces the tensor itself."""
    from fp8_gemms_b200 import _lib, api
    x, res = draw((M, W), BF, 71), draw((M, W), BF, 72)
    w, b = vector(W, BF, 73, 0.2, 1.0), vector(W, BF, 74)
    for fused in (False, True):
        amax = torch.zeros(1, device="cuda")
        if fused:
            y = api.dropout_add_layernorm(x, res, w, b, 0.1, api.dropout_rng(3), amax_out=amax)[1]
        else:
            y = api.layernorm(x, w, b, amax_out=amax)[0]
        q, _, sc = api.cast(y, api.E4M3, amax_in=amax, want_qT=False)
        q2, _, sc2 = api.cast(y, api.E4M3, want_qT=False)
        torch.cuda.synchronize()
        assert torch.equal(q, q2) and torch.equal(sc, sc2)
        assert _lib.lm_get_error()[0] == 0


@pytest.mark.parametrize("rows,cols,dtype", [(300, 1024, BF), (300, 1016, BF), (33, 777, BF),
                                             (65, 4096, BF), (40, 264, torch.float32)])
def test_fused_calls_give_what_the_separate_ones_give(rows, cols, dtype):
    """The forward bit for bit.  The backward's dresidual is dx + ds before dx is rounded, the
    separate sum after it: one rounding of dx apart."""
    from fp8_gemms_b200 import api
    x, r, dy, ds = (draw((rows, cols), dtype, 81 + i) for i in range(4))
    w, b = vector(cols, dtype, 85, 0.2, 1.0), vector(cols, dtype, 86)
    rng = api.dropout_rng(9)
    s, y, mean, rstd = api.dropout_add_layernorm(x, r, w, b, 0.3, rng, 4)
    assert torch.equal(s, api.dropout_add(x, 0.3, rng, 4, residual=r))
    for got, want in zip((y, mean, rstd), api.layernorm(s, w, b)):
        assert torch.equal(got, want)
    dx, dr, dw, db = api.dropout_add_layernorm_backward(dy, ds, s, w, mean, rstd, 0.3, rng, 4)
    one, dw1, db1 = api.layernorm_backward(dy, s, w, mean, rstd)
    assert torch.equal(dw, dw1) and torch.equal(db, db1)
    apart = ref.HALF[dtype] * (np.abs(f64(one)) + np.abs(f64(dr))) + 4 * ref.U * (
        np.abs(f64(one)) + np.abs(f64(ds)))
    close(f64(dr), f64(one) + f64(ds), apart, "dresidual")
    none = api.dropout_add_layernorm_backward(dy, None, s, w, mean, rstd, 0.3, rng, 4)
    assert torch.equal(none[1], one)


def test_two_backward_passes_at_once_on_two_streams():
    """Each call has a workspace of its own."""
    from fp8_gemms_b200 import api
    sets = []
    for k in range(2):
        x, dy = draw((2000, 1024), BF, 91 + 2 * k), draw((2000, 1024), BF, 92 + 2 * k)
        w = vector(1024, BF, 95, 0.2, 1.0)
        _, mean, rstd = api.layernorm(x, w)
        sets.append((dy, x, w, mean, rstd))
    want = [[t.clone() for t in api.layernorm_backward(*a)] for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = [api.layernorm_backward(*a, stream=st) for a, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)
