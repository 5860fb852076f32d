"""The operators' Python calls (csrc/binding.cpp) and the C interface's mirrors in _lib give
the same bits, also from two threads at once, each on a stream of its own; what a call is
given is left alive and unchanged."""
import gc
import sys
import threading

import pytest
import torch

from rows_ref import draw, vector

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROWS, COLS, B, S, H, D = 24, 200, 3, 8, 2, 40


def step(seed, dtype=BF):
    """Every operator once through api; tensors by name, with the arguments."""
    from fp8_gemms_b200 import api
    a = {n: draw((ROWS, COLS), dtype, seed + i) for i, n in enumerate(("x", "res", "dy", "ds"))}
    a["w"], a["b"] = vector(COLS, dtype, seed + 5, 0.2, 1.0), vector(COLS, dtype, seed + 6, 0.1)
    a["q"], a["k"] = (draw((B * S, h * D), dtype, seed + 7 + h).view(B, S, h, D)
                        for h in (H, 1))
    rng = api.dropout_rng(seed, 3)
    freq, mag = api.rope_frequencies(32)
    t = {}
    t["y"], t["mean"], t["rstd"] = api.layernorm(a["x"], a["w"], a["b"])
    t["dx"], t["dw"], t["db"] = api.layernorm_backward(a["dy"], a["x"], a["w"], t["mean"], t["rstd"])
    t["d"] = api.dropout_add(a["x"], 0.3, rng, 2, residual=a["res"])
    t["dd"] = api.dropout_add_backward(a["dy"], 0.3, rng, 2)
    t["s"], t["fy"], t["fm"], t["fr"] = api.dropout_add_layernorm(a["x"], a["res"], a["w"], a["b"],
                                                                  0.3, rng, 2)
    t["fdx"], t["fdr"], t["fdw"], t["fdb"] = api.dropout_add_layernorm_backward(
        a["dy"], a["ds"], t["s"], a["w"], t["fm"], t["fr"], 0.3, rng, 2)
    t["rq"], t["rk"] = api.rope([a["q"], a["k"]], freq, start=5, magnitude=mag)
    t["drq"], = api.rope_backward([a["q"]], freq, start=5, interleaved=True)
    return t, a, rng, freq


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_calls_equal_the_mirrors(dtype):
    from fp8_gemms_b200 import _lib
    t, a, rng, freq = step(11, dtype)
    keep = {n: v.clone() for n, v in a.items()}
    u = {n: torch.full_like(v, 7.0) for n, v in t.items()}
    ws = torch.empty(_lib.lm_layernorm_workspace_size(ROWS, COLS), dtype=torch.uint8, device="cuda")
    _lib.lm_layernorm_fwd(a["x"], a["w"], a["b"], u["y"], u["mean"], u["rstd"])
    _lib.lm_layernorm_bwd(a["dy"], a["x"], a["w"], u["mean"], u["rstd"], u["dx"], u["dw"], u["db"],
                          ws)
    _lib.lm_dropout_add_fwd(a["x"], a["res"], u["d"], 0.3, rng, 2)
    _lib.lm_dropout_add_bwd(a["dy"], u["dd"], 0.3, rng, 2)
    _lib.lm_dropout_add_layernorm_fwd(a["x"], a["res"], a["w"], a["b"], u["s"], u["fy"], 0.3, rng,
                                      2, u["fm"], u["fr"])
    _lib.lm_dropout_add_layernorm_bwd(a["dy"], a["ds"], u["s"], a["w"], u["fm"], u["fr"], 0.3, rng,
                                      u["fdx"], u["fdr"], u["fdw"], u["fdb"], ws, offset=2)
    _lib.lm_rope([a["q"], a["k"]], [u["rq"], u["rk"]], freq, start=5)
    _lib.lm_rope([a["q"]], [u["drq"]], freq, start=5,
                 flags=_lib.ROPE_INTERLEAVED | _lib.ROPE_INVERSE)
    for n in t:
        assert torch.equal(t[n], u[n]), n
    for n in a:
        assert torch.equal(a[n], keep[n]), n


def test_two_threads_on_two_streams():
    want = [step(s)[0] for s in (21, 22)]
    torch.cuda.synchronize()
    bad, errors = [], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = step(21 + i)[0]
                    bad.extend(n for n in got if not torch.equal(got[n], want[i][n]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors and not bad


def test_calls_keep_no_reference():
    """Also refused calls: nothing they were given stays alive after them."""
    from fp8_gemms_b200 import api
    x, w, q = draw((4, 64), BF, 1), vector(64, BF, 2), draw((2, 8), BF, 3).view(1, 2, 1, 8)
    freq, _ = api.rope_frequencies(8)
    rng, out, xs = api.dropout_rng(1), torch.empty_like(q), [q]
    args = (x, w, q, freq, rng, out, xs)
    before = [sys.getrefcount(v) for v in args]
    for _ in range(3):
        api.layernorm(x, w)
        api.dropout_add(x, 0.1, rng, residual=x)
        got = api.rope(xs, freq, out=[out])
        assert got[0] is out
        del got
        for call in (lambda: api.layernorm(x, w[:63]), lambda: api.dropout_add(x, 1.5, rng),
                     lambda: api.rope(xs, freq, out=[x])):
            with pytest.raises(api.LmError):
                call()
    gc.collect()
    assert [sys.getrefcount(v) for v in args] == before
