"""The operators between the GEMMs of a training block, as they are measured:

- layer norm, forward and backward ("ln");
- dropout from a counter-based generator, added to the residual stream,
  forward and backward ("dropout");
- the two in one pass, s = residual + dropout(x), y = LN(s), forward and
  backward ("dropout_ln");
- rotary positions of the Q and K projections, forward and backward ("rope").

With `own` false, run() computes them in elementary torch operations; with
`own` true, through fp8_gemms_b200.api.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the norm of a handful of rows: one short evaluation prompt, where latency counts
        _ln("ln_fwd_few_rows", "fwd", 16, 1024, "bf16"),
        # a training micro-batch of 16384 tokens
        _ln("ln_fwd_batch", "fwd", 16384, 4096, "bf16"),
        _ln("ln_bwd_batch", "bwd", 16384, 4096, "bf16"),
        # an fp32 block whose width is no multiple of anything
        _ln("ln_bwd_odd_fp32", "bwd", 2051, 1537, "fp32"),
        # dropout of the MLP's hidden activations, f = 12288: the largest
        _drop("dropout_bwd_hidden", "bwd", 16384, 12288, "bf16", 0.1, False),
        # a ragged batch whose rows start at every alignment
        _drop("dropout_fwd_odd", "fwd", 1999, 1001, "bf16", 0.3, True),
        # the end of a branch and the norm of the next, a micro-batch
        _drop_ln("dropout_ln_fwd_batch", "fwd", 8192, 5120, "bf16", 0.1),
        _drop_ln("dropout_ln_bwd_batch", "bwd", 8192, 8192, "bf16", 0.1),
        # the same in fp32 for a small model and a short batch
        _drop_ln("dropout_ln_fwd_small_fp32", "fwd", 128, 768, "fp32", 0.2),
        # one new token for each of 64 sequences, far into a long context
        _rope("rope_decode", "fwd", 64, 1, 24, 8, 128, 128, "bf16", "half", "bshd", 100003, 8.0),
        # the Q and K projections of a micro-batch of 8 x 2048 tokens, 24 + 8 heads of 128
        _rope("rope_batch", "fwd", 8, 2048, 24, 8, 128, 128, "bf16", "half", "bshd", 0, 1.0),
        # rotation of 32 of 80 elements, neighbours paired, heads before tokens, a ragged length
        _rope("rope_bwd_partial_fp32", "bwd", 3, 1333, 12, 12, 80, 32, "fp32", "interleaved",
              "bhsd", 0, 1.0),
    ]


def _ln(name, direction, rows, cols, dtype):
    return {"name": name, "op": "ln", "dir": direction, "rows": rows, "cols": cols,
            "dtype": dtype}


def _drop(name, direction, rows, cols, dtype, p, residual):
    return {"name": name, "op": "dropout", "dir": direction, "rows": rows, "cols": cols,
            "dtype": dtype, "p": p, "residual": residual}


def _drop_ln(name, direction, rows, cols, dtype, p):
    return {"name": name, "op": "dropout_ln", "dir": direction, "rows": rows, "cols": cols,
            "dtype": dtype, "p": p}


def _rope(name, direction, batch, seq, q_heads, kv_heads, head_dim, rot_dim, dtype, pairs,
          layout, start, stretch):
    """pairs: "half" (i with i + rot/2) or "interleaved" (2i with 2i + 1).
    layout: "bshd", "bhsd", or "qkv" (Q and K are slices of one [b, s, q+2kv, d]
    projection).  start: the first token's position.  stretch > 1: the
    frequencies are scaled by parts for a context that many times longer."""
    return {"name": name, "op": "rope", "dir": direction, "batch": batch, "seq": seq,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "rot_dim": rot_dim,
            "dtype": dtype, "pairs": pairs, "layout": layout, "start": start,
            "stretch": stretch}


MOST_BYTES = 2 * 16384 * 12288 * 2     # of the largest listed case


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(["ln", "dropout", "dropout_ln", "rope"])
        direction = rng.choice(["fwd", "bwd"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if op == "rope":
            kv = rng.choice([1, 2, 3, 8, 12])
            head_dim = rng.choice([32, 48, 64, 80, 96, 100, 128, 192, 256])
            rot = rng.choice([head_dim, head_dim, 2 * rng.randint(1, head_dim // 2)])
            case = _rope("", direction, rng.randint(1, 16), _log_uniform(rng, 1, 8192),
                         kv * rng.randint(1, 8), kv, head_dim, rot, dtype,
                         rng.choice(["half", "interleaved"]),
                         rng.choice(["bshd", "bhsd", "qkv"]),
                         rng.choice([0, rng.randint(1, 1 << 20)]),
                         rng.choice([1.0, rng.uniform(1.5, 32.0)]))
        else:
            rows, cols = _log_uniform(rng, 1, 16384), _log_uniform(rng, 16, 16384)
            # every second width is one that a model has, the others fall where they fall
            if rng.random() < 0.5:
                cols = max(64, cols // 64 * 64)
            p = rng.choice([0.05, 0.1, 0.2, 0.5, rng.uniform(0.01, 0.6)])
            case = {"ln": lambda: _ln("", direction, rows, cols, dtype),
                    "dropout": lambda: _drop("", direction, rows, cols, dtype, p,
                                             direction == "fwd" and rng.random() < 0.7),
                    "dropout_ln": lambda: _drop_ln("", direction, rows, cols, dtype, p)}[op]()
        del case["name"]
        if work(case)["bytes"] <= MOST_BYTES:
            return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        tokens = case["batch"] * case["seq"]
        heads = case["q_heads"] + case["kv_heads"]
        n = tokens * heads * case["head_dim"]
        return {"bytes": 2 * n * e + 8 * tokens + 4 * case["rot_dim"],
                "flops": 3 * tokens * heads * case["rot_dim"]}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * n * e,
                "flops": (2 if case["residual"] else 1) * n}
    small = 8 * rows + 2 * cols * e              # mean and rstd; weight and bias or weight
    if case["dir"] == "bwd":
        small += cols * e                        # weight in, dweight and dbias out
    passes, flops = {("ln", "fwd"): (2, 8), ("ln", "bwd"): (3, 14),
                     ("dropout_ln", "fwd"): (4, 10), ("dropout_ln", "bwd"): (5, 16)}[
                         case["op"], case["dir"]]
    return {"bytes": passes * n * e + small, "flops": flops * n}


# --------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, device="cuda").normal_(mean, sigma, generator=gen).to(dtype)

    st = {"case": dict(case)}
    if case["op"] == "rope":
        return _prepare_rope(case, st, normal, gen)
    rows, cols = case["rows"], case["cols"]
    if case["op"] != "dropout":
        st["weight"] = normal(cols, sigma=0.2, mean=1.0)
        st["bias"] = normal(cols, sigma=0.1)
    if case["op"] != "ln":
        # {seed, offset} on the device, as a training loop keeps and advances it
        st["rng"] = torch.randint(0, 1 << 62, (2,), device="cuda", generator=gen)
    if case["dir"] == "fwd":
        st["x"] = normal(rows, cols, sigma=0.7, mean=0.1)
        if case["op"] == "dropout_ln" or case.get("residual"):
            st["residual"] = normal(rows, cols, sigma=2.0, mean=-0.2)
        return st
    st["dy"] = normal(rows, cols, sigma=1e-2)
    if case["op"] != "dropout":
        # the forward's input and what it saved
        x = normal(rows, cols, sigma=2.0, mean=0.2)
        x64 = x.double()
        mean = x64.mean(1)
        var = ((x64 - mean[:, None]) ** 2).mean(1)
        st["x"], st["mean"] = x, mean.float()
        st["rstd"] = (1.0 / torch.sqrt(var + EPS)).float()
    if case["op"] == "dropout_ln":
        st["ds"] = normal(rows, cols, sigma=1e-2)
    return st


def _prepare_rope(case, st, normal, gen):
    b, s, hq, hk, d = (case[k] for k in ("batch", "seq", "q_heads", "kv_heads", "head_dim"))
    if case["layout"] == "qkv":
        qkv = normal(b, s, hq + 2 * hk, d)
        st["q"], st["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    elif case["layout"] == "bhsd":
        # stored heads first; seen as [batch, seq, head, dim]
        st["q"] = normal(b, hq, s, d).transpose(1, 2)
        st["k"] = normal(b, hk, s, d).transpose(1, 2)
    else:
        st["q"], st["k"] = normal(b, s, hq, d), normal(b, s, hk, d)
    # every sequence of the batch is at a place of its own
    first = torch.randint(0, 4096, (b, 1), device="cuda", generator=gen)
    st["positions"] = case["start"] + first + torch.arange(s, device="cuda")[None, :]
    st["inv_freq"], st["magnitude"] = _frequencies(case["rot_dim"], case["stretch"])
    return st


def _frequencies(rot_dim, stretch, theta=10000.0, context=2048, slow=1.0, fast=32.0):
    """Inverse frequencies in 64 bits and the magnitude.  With stretch > 1, those
    that turn less than `slow` times over the original context are divided by
    stretch, those that turn more than `fast` times stay, and the ones between
    are blended; the magnitude is 0.1 ln(stretch) + 1."""
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = theta ** (-i / rot_dim)
    if stretch > 1.0:
        turns = context * f / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f / stretch * (1.0 - keep) + f * keep
    return f.cuda(), 0.1 * math.log(stretch) + 1.0 if stretch > 1.0 else 1.0


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        return _own(st, case)
    return {"ln": _plain_ln, "dropout": _plain_dropout, "dropout_ln": _plain_dropout_ln,
            "rope": _plain_rope}[case["op"]](st, case)


def _own(st, case):
    from fp8_gemms_b200 import api
    op, fwd = case["op"], case["dir"] == "fwd"
    if op == "ln":
        if fwd:
            return api.layernorm(st["x"], st["weight"], st["bias"], eps=EPS)
        return api.layernorm_backward(st["dy"], st["x"], st["weight"], st["mean"], st["rstd"])
    if op == "dropout":
        if fwd:
            return api.dropout_add(st["x"], case["p"], st["rng"], residual=st.get("residual"))
        return api.dropout_add_backward(st["dy"], case["p"], st["rng"])
    if op == "dropout_ln":
        if fwd:
            return api.dropout_add_layernorm(st["x"], st["residual"], st["weight"], st["bias"],
                                             case["p"], st["rng"], eps=EPS)
        return api.dropout_add_layernorm_backward(st["dy"], st["ds"], st["x"], st["weight"],
                                                  st["mean"], st["rstd"], case["p"], st["rng"])
    call = api.rope if fwd else api.rope_backward
    return call([st["q"], st["k"]], st["inv_freq"], positions=st["positions"],
                interleaved=case["pairs"] == "interleaved", magnitude=st["magnitude"])


# ------------------------------------------------------------ the plain forms
def _plain_norm(x, weight, bias):
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)
    return (x - mean) * rstd * weight.float() + bias.float(), mean[:, 0], rstd[:, 0]


def _plain_norm_grads(dy, x, weight, mean, rstd):
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy * weight.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


def _plain_ln(st, case):
    dt = DTYPES[case["dtype"]]
    if case["dir"] == "fwd":
        y, mean, rstd = _plain_norm(st["x"].float(), st["weight"], st["bias"])
        return y.to(dt), mean, rstd
    return tuple(t.to(dt) for t in _plain_norm_grads(
        st["dy"].float(), st["x"].float(), st["weight"], st["mean"], st["rstd"]))


def _mulhilo(a, m):
    """High and low 32 bits of a * m, both below 2^32, in int64 (which wraps)."""
    prod = a * m
    return (prod >> 32) & 0xFFFFFFFF, prod & 0xFFFFFFFF


def _keep(rows, cols, p, rng):
    """Which elements stay, and the factor of those.  Element (r, c) has the 16
    bits c % 8 of Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy
    as 1, 2, 3", 2011) at counter {c / 8, r, offset} under the key `seed`."""
    groups = -(-cols // 8)
    seed, offset = rng[0], rng[1]
    c0 = torch.arange(groups, device=rng.device)[None, :].expand(rows, groups)
    c1 = torch.arange(rows, device=rng.device)[:, None].expand(rows, groups)
    c2 = (offset & 0xFFFFFFFF).expand(rows, groups)
    c3 = ((offset >> 32) & 0xFFFFFFFF).expand(rows, groups)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16,
                         c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], dim=2)
    drop = round(p * 65536)
    scale = 65536.0 / (65536 - drop)
    return words.reshape(rows, groups * 8)[:, :cols] >= drop, scale


def _dropped(x, keep, scale):
    return torch.where(keep, x * scale, 0.0)


def _plain_dropout(st, case):
    x = st["x"] if case["dir"] == "fwd" else st["dy"]
    keep, scale = _keep(case["rows"], case["cols"], case["p"], st["rng"])
    y = _dropped(x.float(), keep, scale)
    if "residual" in st:
        y = st["residual"].float() + y
    return y.to(x.dtype)


def _plain_dropout_ln(st, case):
    dt = DTYPES[case["dtype"]]
    keep, scale = _keep(case["rows"], case["cols"], case["p"], st["rng"])
    if case["dir"] == "fwd":
        s = (st["residual"].float() + _dropped(st["x"].float(), keep, scale)).to(dt)
        # the norm is that of the stream as it is stored
        y, mean, rstd = _plain_norm(s.float(), st["weight"], st["bias"])
        return s, y.to(dt), mean, rstd
    dx, dweight, dbias = _plain_norm_grads(st["dy"].float(), st["x"].float(), st["weight"],
                                           st["mean"], st["rstd"])
    total = st["ds"].float() + dx
    return tuple(t.to(dt) for t in (_dropped(total, keep, scale), total, dweight, dbias))


def _plain_rope(st, case):
    # the angles of far positions in 64 bits
    angle = st["positions"].double()[:, :, None] * st["inv_freq"]
    cos = (torch.cos(angle) * st["magnitude"]).float()[:, :, None, :]
    sin = (torch.sin(angle) * st["magnitude"]).float()[:, :, None, :]
    if case["dir"] == "bwd":
        sin = -sin
    return [_plain_rotate(x, cos, sin, case["rot_dim"], case["pairs"] == "interleaved")
            for x in (st["q"], st["k"])]


def _plain_rotate(x, cos, sin, rot, interleaved):
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    y[..., rot:] = x[..., rot:]
    first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
                     else (slice(0, rot // 2), slice(rot // 2, rot)))
    a, b = x[..., first].float(), x[..., second].float()
    y[..., first] = (a * cos - b * sin).to(x.dtype)
    y[..., second] = (b * cos + a * sin).to(x.dtype)
    return y


# ------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    v = {k: t.double() for k, t in st.items()
         if torch.is_tensor(t) and t.is_floating_point()}
    if case["op"] == "rope":
        return _exact_rope(case, st)
    fwd = case["dir"] == "fwd"
    factor = _exact_factor(case, st["rng"]) if case["op"] != "ln" else None
    if case["op"] == "dropout":
        return v["x" if fwd else "dy"] * factor + v.get("residual", 0.0)
    if fwd:
        s = v["x"]
        if factor is not None:
            s = (s * factor + v["residual"]).to(DTYPES[case["dtype"]]).double()
        n = s.shape[1]
        mean = s.sum(1) / n
        centred = s - mean[:, None]
        rstd = (torch.einsum("rc,rc->r", centred, centred) / n + EPS).rsqrt()
        y = torch.addcmul(v["bias"], centred * v["weight"], rstd[:, None])
        return (y, mean, rstd) if factor is None else (s, y, mean, rstd)
    # dx = J^T (w dy), J the Jacobian of h: rstd (I - 1 1^T / n - h h^T / n)
    n = v["dy"].shape[1]
    h = v["rstd"][:, None] * (v["x"] - v["mean"][:, None])
    g = v["dy"] * v["weight"]
    along = torch.einsum("rc,rc->r", g, h)[:, None] * h + g.sum(1)[:, None]
    dx = (n * g - along) * (v["rstd"][:, None] / n)
    dweight, dbias = torch.einsum("rc,rc->c", v["dy"], h), v["dy"].sum(0)
    if factor is None:
        return dx, dweight, dbias
    total = dx + v["ds"]
    return total * factor, total, dweight, dbias


def _exact_factor(case, rng):
    """0 or the scale of every element, with the generator's products taken in
    halves of 16 bits."""
    rows, cols = case["rows"], case["cols"]
    low = (1 << 32) - 1
    seed, offset = (int(t) for t in rng.tolist())

    def product(a, m):
        m0, m1 = m & 0xFFFF, m >> 16
        a0, a1 = a & 0xFFFF, a >> 16
        mid = a1 * m0 + ((a0 * m0) >> 16)
        mid2 = a0 * m1 + (mid & 0xFFFF)
        return a1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 << 16) | (a0 * m0 & 0xFFFF)) & low

    shape = (rows, (cols + 7) // 8)
    state = [torch.zeros(shape, dtype=torch.int64, device=rng.device) for _ in range(4)]
    state[0] += torch.arange(shape[1], device=rng.device)
    state[1] += torch.arange(rows, device=rng.device).unsqueeze(1)
    state[2] += offset & low
    state[3] += (offset >> 32) & low
    for r in range(10):
        key = [((seed & low) + r * 0x9E3779B9) & low, ((seed >> 32) + r * 0xBB67AE85) & low]
        hi_a, lo_a = product(state[0], 0xD2511F53)
        hi_b, lo_b = product(state[2], 0xCD9E8D57)
        state = [hi_b ^ state[1] ^ key[0], lo_b, hi_a ^ state[3] ^ key[1], lo_a]
    drop = round(case["p"] * 65536)
    out = torch.zeros(rows, shape[1] * 8, dtype=torch.float64, device=rng.device)
    for j in range(8):
        out[:, j::8] = ((state[j // 2] >> (16 * (j % 2))) & 0xFFFF >= drop).double()
    return out[:, :cols] * (65536.0 / (65536 - drop))


def _exact_rope(case, st):
    turn = torch.polar(torch.full_like(st["positions"], st["magnitude"], dtype=torch.float64)
                       [:, :, None].expand(-1, -1, case["rot_dim"] // 2),
                       st["positions"].double()[:, :, None] * st["inv_freq"])
    if case["dir"] == "bwd":
        turn = turn.conj()
    rot, outs = case["rot_dim"], []
    for x in (st["q"].double(), st["k"].double()):
        head = x[..., :rot].contiguous()
        if case["pairs"] == "half":
            head = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2).contiguous()
        else:
            head = head.unflatten(-1, (rot // 2, 2))
        head = torch.view_as_real(torch.view_as_complex(head) * turn[:, :, None, :])
        if case["pairs"] == "half":
            head = head.transpose(-1, -2)
        outs.append(torch.cat([head.flatten(-2), x[..., rot:]], dim=-1))
    return outs
