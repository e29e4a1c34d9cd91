"""The layer operators' cases: what is timed, on what inputs, and their plain forms.

The operators are those that a training step runs around the optimizer step of
this package, on activations kept in 8 bits:

  ckpt    an activation saved in 8 bits and loaded again
  fwd     the norms after and before a block, with gate and residual scale,
          where nothing is kept for a backward pass
  bwd     their backward pass, from 8-bit checkpoints
  site    both in one training pass; the checkpoints are the forward's own
  wgrad   weight gradients of linear layers, from the saved inputs: the
          gradients the optimizer step reads

Checkpoint format. A row is cut into groups of 32 columns (the last may be
shorter). A group holds one exponent byte E and one byte per element; an
element's value is q * 2^(E-127), q an int8 in [-127, 127] or an e4m3 number.
2^(E-127) is the smallest power of two (at least 2^-110) with
max|x| <= 127 * 2^(E-127) (int8) or 448 * 2^(E-127) (e4m3), and q is
x / 2^(E-127) rounded to nearest, ties to even. A group that holds an infinity
or a NaN has E = 255 and stands for NaNs. Rows are padded to a multiple of 16
bytes (q) and hold ceil(cols / 32) exponent bytes (e).
"""
import torch

own = False

GROUP = 32
TOP = {"int8": 127.0, "e4m3": 448.0}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # One token's hidden state of the 1.7B layer: the smallest call, all latency.
        {"name": "ckpt_token", "op": "ckpt", "rows": 1, "cols": 2048, "dtype": "bf16", "kind": "int8"},
        # Odd sizes in fp32 and the wide-range element type: a ragged last group, unaligned rows.
        {"name": "ckpt_ragged_f32", "op": "ckpt", "rows": 1001, "cols": 1111, "dtype": "f32", "kind": "e4m3"},
        # The input of the down projection of the 32B layer, one sequence: the largest activation of a layer.
        {"name": "ckpt_mlp", "op": "ckpt", "rows": 4096, "cols": 25600, "dtype": "bf16", "kind": "int8"},
        # A norm site of the 32B layer, one token, in evaluation.
        {"name": "fwd_token", "op": "fwd", "rows": 1, "cols": 5120, "dtype": "bf16", "post": True, "gate": "feature"},
        # The same site over one sequence, in evaluation.
        {"name": "fwd_sequence", "op": "fwd", "rows": 4096, "cols": 5120, "dtype": "bf16", "post": True, "gate": "feature"},
        # The same site in training: forward with its checkpoints, then backward from them.
        {"name": "site_sequence", "op": "site", "rows": 4096, "cols": 5120, "dtype": "bf16", "kind": "int8", "post": True, "gate": "feature"},
        # Backward of a few tokens in fp32 with odd sizes and a gate per token and feature.
        {"name": "bwd_ragged_f32", "op": "bwd", "rows": 37, "cols": 201, "dtype": "f32", "kind": "e4m3", "post": True, "gate": "token"},
        # Backward of a site of the 1.7B layer over four sequences.
        {"name": "bwd_batch", "op": "bwd", "rows": 16384, "cols": 2048, "dtype": "bf16", "kind": "int8", "post": True, "gate": "feature"},
        # Weight gradient of a small layer in fp32 over a few tokens: latency, odd sizes.
        {"name": "wgrad_small_f32", "op": "wgrad", "rows": 101, "shapes": "203x137", "dtype": "f32", "gdtype": "f32", "kind": "int8", "scale": True, "beta": 0.0},
        # The k projection of the 32B layer, accumulated into an fp32 gradient over micro batches: few tiles, a long sum.
        {"name": "wgrad_k_accumulate", "op": "wgrad", "rows": 4096, "shapes": "1024x5120", "dtype": "bf16", "gdtype": "f32", "kind": "int8", "scale": True, "beta": 1.0},
        # All seven matrices of the 1.7B layer, one sequence ('|' separates inputs; q, k, v share one, gate and up another).
        {"name": "wgrad_layer", "op": "wgrad", "rows": 4096, "shapes": "2048x2048 1024x2048 1024x2048|2048x2048|6144x2048 6144x2048|2048x6144",
         "dtype": "bf16", "gdtype": "bf16", "kind": "int8", "scale": False, "beta": 0.0},
        # One MLP matrix of the 32B layer over two sequences: the largest product.
        {"name": "wgrad_mlp", "op": "wgrad", "rows": 8192, "shapes": "25600x5120", "dtype": "bf16", "gdtype": "bf16", "kind": "e4m3", "scale": True, "beta": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["ckpt", "fwd", "bwd", "site", "wgrad", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kind = rng.choice(["int8", "e4m3"])
    even = rng.choice([1, 8, 64])  # odd sizes as often as aligned ones
    if op == "wgrad":
        rows = _log(rng, 1, 8192)
        shapes = []
        for _ in range(rng.choice([1, 1, 2, 3])):
            shapes.append("%dx%d" % tuple(max(even, _log(rng, 16, 6000) // even * even) for _ in range(2)))
        sep = rng.choice(["|", "|", " "])
        if sep == " ":  # one shared input: one width
            shapes = [s.split("x")[0] + "x" + shapes[0].split("x")[1] for s in shapes]
        return {"op": op, "rows": rows, "shapes": sep.join(shapes), "dtype": dtype, "gdtype": rng.choice(["f32", dtype]), "kind": kind,
                "scale": rng.random() < 0.5, "beta": rng.choice([0.0, 0.0, 1.0])}
    rows = _log(rng, 1, 8192)
    cols = max(even, _log(rng, 32, 25600 if op == "ckpt" else 8192) // even * even)
    case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype}
    if op != "fwd":
        case["kind"] = kind
    if op == "site":
        case["dtype"] = "bf16"  # in fp32 a rounding border crossed by the last bit of a norm would show in every gradient
    if op != "ckpt":
        case["post"] = rng.random() < 0.75
        case["gate"] = rng.choice(["feature", "token", "none"])
    return case


# ------------------------------------------------------------------ the format


def _pow2(k):
    """2^k in fp32, exactly, for -126 <= k <= 127."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x, kind):
    """(q bytes [rows, padded], e bytes [rows, groups]) of x [rows, cols]."""
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    x = torch.nn.functional.pad(x.float(), (0, groups * GROUP - cols)).view(rows, groups, GROUP)
    top = x.abs().amax(2)
    fine = torch.isfinite(x).all(2)
    top = torch.where(fine, top, torch.zeros_like(top))
    # m * 2^k with m in [1/2, 1): the smallest e with m * 2^k <= TOP * 2^e
    m, k = torch.frexp(top)
    e = torch.where(m <= TOP[kind] / 2.0 ** (7 if kind == "int8" else 9), k - (7 if kind == "int8" else 9), k - (6 if kind == "int8" else 8))
    e = torch.where(top == 0, torch.full_like(e, -110), e).clamp(min=-110)
    y = torch.where(fine[..., None], x * _pow2(-e)[..., None], torch.zeros_like(x))
    if kind == "int8":
        q = torch.round(y).to(torch.int8).view(torch.uint8)
    else:
        q = y.to(torch.float8_e4m3fn).view(torch.uint8)
    q = q.view(rows, groups * GROUP)[:, :cols]
    q = torch.nn.functional.pad(q, (0, -cols % 16)).contiguous()
    e = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return q, e


def _values(q, e, cols, kind):
    """The fp32 values that a checkpoint stands for."""
    v = q[:, :cols]
    v = v.view(torch.int8).float() if kind == "int8" else v.view(torch.float8_e4m3fn).float()
    unit = torch.where(e == 255, torch.full((), float("nan"), device=e.device), _pow2(e.to(torch.int32).clamp(max=254) - 127))
    return v * unit.repeat_interleave(GROUP, 1)[:, :cols]


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, cols, dtype):
    """Hidden states: normal, with a scale per token and a few loud channels."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= 1 + 15 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    return x.to(DT[dtype])


def _shapes(case):
    return [[tuple(int(v) for v in s.split("x")) for s in part.split()] for part in case["shapes"].split("|")]


def prepare(case, seed):
    g = _gen(seed)
    op, rows, dt = case["op"], case["rows"], DT[case["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if op == "ckpt":
        st["x"] = _activations(g, rows, case["cols"], case["dtype"])
        st["out"] = torch.empty_like(st["x"])
    elif op == "wgrad":
        st["dy"], st["in"], st["g"], st["scale"] = [], [], [], []
        for part in _shapes(case):
            cols = part[0][1]
            x = _activations(g, rows, cols, "f32")
            q, e = _quantise(x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS), case["kind"])
            scale = (1 + 0.1 * rand(cols)).to(dt) if case["scale"] else None
            for n, _ in part:
                st["dy"].append((1e-3 * rand(rows, n)).to(dt))
                st["in"].append((q, e))
                st["scale"].append(scale)
                st["g"].append(torch.empty(n, cols, dtype=DT[case["gdtype"]], device="cuda"))
        # what earlier micro batches left
        st["g0"] = [(1e-2 * rand(*t.shape)).to(t.dtype) if case["beta"] else None for t in st["g"]]
    else:
        cols = case["cols"]
        st["r"] = _activations(g, rows, cols, case["dtype"])
        st["b"] = _activations(g, rows, cols, case["dtype"])
        st["w_pre"] = (1 + 0.1 * rand(cols)).to(dt)
        st["w_post"] = (1 + 0.1 * rand(cols)).to(dt) if case["post"] else None
        st["gate"] = None if case["gate"] == "none" else (0.5 + 0.2 * (rand(cols) if case["gate"] == "feature" else rand(rows, cols))).to(dt)
        st["res_scale"], st["branch_scale"] = 0.9, 0.7
        if op != "fwd":
            st["dy"] = (1e-3 * rand(rows, cols)).to(dt)
            st["dh"] = (1e-3 * rand(rows, cols)).to(dt)
        if op == "bwd":
            f = _forward(st, torch.float32)
            st["rstd_y"], st["rstd_b"] = f["rstd_y"], f["rstd_b"]
            st["u"], st["v"] = _quantise(f["u"], case["kind"]), _quantise(f["v"], case["kind"])
    if own:
        _handles(st)
    return st


def _handles(st):
    """What a program keeps between passes: buffers for the results, and the call's descriptors."""
    from matrix_optimizer_step_muon_amd import layer
    case, rows = st["case"], st["case"]["rows"]
    if case["op"] == "ckpt":
        st["q8"] = layer.Q8(rows, case["cols"], case["kind"])
    elif case["op"] == "wgrad":
        saved = {id(q): layer.Q8(rows, part[0][1], case["kind"], q=q, e=e)
                 for part, (q, e) in zip([p for p in _shapes(case) for _ in p], st["in"])}
        st["plan"] = layer.WGrad([(dy, saved[id(q)], g, s, case["beta"], g0)
                                  for dy, (q, _), g, s, g0 in zip(st["dy"], st["in"], st["g"], st["scale"], st["g0"])])
    else:
        saved = None
        if case["op"] == "bwd":
            saved = (layer.Q8(rows, case["cols"], case["kind"], q=st["u"][0], e=st["u"][1]),
                     layer.Q8(rows, case["cols"], case["kind"], q=st["v"][0], e=st["v"][1]), st["rstd_y"], st["rstd_b"])
        st["site"] = layer.NormSite(st["b"], st["r"], st["w_pre"], w_post=st["w_post"], gate=st["gate"], res_scale=st["res_scale"],
                                    branch_scale=st["branch_scale"], eps=EPS, kind=case.get("kind"), saved=saved)


# ------------------------------------------------------------------ one pass


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    from matrix_optimizer_step_muon_amd import layer
    op = st["case"]["op"]
    if op == "ckpt":
        layer.q8_save(st["x"], st["q8"])
        layer.q8_load(st["q8"], st["out"])
        return st["out"]
    if op == "wgrad":
        st["plan"].run()
        return list(st["g"])
    site, out = st["site"], {}
    if op != "bwd":
        site.forward()
        out = {"y": site.y, "h": site.h}
    if op != "fwd":
        site.backward(st["dy"], st["dh"])
        out.update({"d_residual": site.d_residual, "d_branch": site.d_branch, "d_w_pre": site.d_w_pre,
                    "d_w_post": site.d_w_post, "d_gate": site.d_gate})
    return out


def _forward(st, t):
    """y, h and what a backward pass needs of them, in the type t."""
    b, r, w_pre = st["b"].to(t), st["r"].to(t), st["w_pre"].to(t)
    out = {"v": b, "rstd_b": None}
    if st["w_post"] is not None:
        out["rstd_b"] = torch.rsqrt(b.square().mean(1) + EPS)
        out["v"] = b * out["rstd_b"][:, None]
    n = out["v"] if st["w_post"] is None else out["v"] * st["w_post"].to(t)
    if st["gate"] is not None:
        n = n * st["gate"].to(t)
    out["y"] = st["res_scale"] * r + st["branch_scale"] * n
    out["rstd_y"] = torch.rsqrt(out["y"].square().mean(1) + EPS)
    out["u"] = out["y"] * out["rstd_y"][:, None]
    out["h"] = out["u"] * w_pre
    return out


def _backward(st, u, v, rstd_y, rstd_b, t):
    """The gradients, in the type t, from the values u and v that the checkpoints stand for."""
    dh = st["dh"].to(t)
    du = dh * st["w_pre"].to(t)
    s = st["dy"].to(t) + rstd_y.to(t)[:, None] * (du - u * (du * u).mean(1, keepdim=True))
    out = {"d_residual": st["res_scale"] * s, "d_w_pre": (dh * u).sum(0), "d_w_post": None, "d_gate": None}
    dn = st["branch_scale"] * s
    if st["gate"] is not None:
        out["d_gate"] = dn * (v if st["w_post"] is None else v * st["w_post"].to(t))
        if st["gate"].dim() == 1:
            out["d_gate"] = out["d_gate"].sum(0)
        dn = dn * st["gate"].to(t)
    if st["w_post"] is not None:
        out["d_w_post"] = (dn * v).sum(0)
        dv = dn * st["w_post"].to(t)
        dn = rstd_b.to(t)[:, None] * (dv - v * (dv * v).mean(1, keepdim=True))
    out["d_branch"] = dn
    return out


def _run_plain(st):
    case = st["case"]
    dt = DT[case["dtype"]]
    cast = lambda d: {k: None if x is None else x.to(dt) for k, x in d.items()}  # noqa: E731
    if case["op"] == "ckpt":
        q, e = _quantise(st["x"], case["kind"])
        return _values(q, e, case["cols"], case["kind"]).to(dt)
    if case["op"] == "wgrad":
        return [_product(dy, _values(q, e, g.shape[1], case["kind"]), s, case["beta"], g0, g.dtype)
                for dy, (q, e), s, g, g0 in zip(st["dy"], st["in"], st["scale"], st["g"], st["g0"])]
    out = {}
    if case["op"] != "bwd":
        f = _forward(st, torch.float32)
        out = cast({"y": f["y"], "h": f["h"]})
        if case["op"] == "site":
            u, v = (_values(*_quantise(f[k], case["kind"]), case["cols"], case["kind"]) for k in ("u", "v"))
            out.update(cast(_backward(st, u, v, f["rstd_y"], f["rstd_b"], torch.float32)))
        return out
    u, v = (_values(*st[k], case["cols"], case["kind"]) for k in ("u", "v"))
    return cast(_backward(st, u, v, st["rstd_y"], st["rstd_b"], torch.float32))


def _product(dy, x, scale, beta, g0, gdt):
    g = dy.float().t() @ x
    if scale is not None:
        g = g * scale.float()
    if g0 is not None:
        g = g + beta * g0.float()
    return g.to(gdt)


# ------------------------------------------------------------------ the work


def work(case):
    """Each input read once, each output written once; the products' flops."""
    rows, b = case["rows"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "wgrad":
        gb = 2 if case["gdtype"] == "bf16" else 4
        by = fl = 0
        for part in _shapes(case):
            cols = part[0][1]
            by += rows * (cols + -(-cols // GROUP)) + (cols * b if case["scale"] else 0)
            for n, _ in part:
                by += rows * n * b + n * cols * gb * (2 if case["beta"] else 1)
                fl += 2 * rows * n * cols
        return {"bytes": by, "flops": fl}
    cols = case["cols"]
    n, q8 = rows * cols, rows * (cols + -(-cols // GROUP))
    if case["op"] == "ckpt":  # x in, the checkpoint out and in again, x out
        return {"bytes": 2 * n * b + 2 * q8, "flops": 4 * n}
    gate = {"none": 0, "feature": cols, "token": n}[case["gate"]]
    weights = cols + (cols if case["post"] else 0) + gate
    by = fl = 0
    if case["op"] in ("fwd", "site"):  # branch and residual in, y and h out (and the checkpoints)
        by += (4 * n + weights) * b + 4 * rows * (2 if case["post"] else 1) + (2 * q8 if case["op"] == "site" else 0)
        fl += 12 * n
    if case["op"] in ("bwd", "site"):  # dy, dh and the checkpoints in, two gradients and the weights' out
        by += (4 * n + 2 * weights) * b + 2 * q8 + 4 * rows * (2 if case["post"] else 1)
        fl += 24 * n
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ in 64 bits


def _two(k):
    """2^k in fp64, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_values(q, e, cols, kind):
    b = q[:, :cols].long()
    if kind == "int8":
        v = torch.where(b < 128, b, b - 256).double()
    else:
        ex, m = (b >> 3) & 15, (b & 7).double()
        v = torch.where(ex == 0, m * 2.0 ** -9, (8 + m) * _two(ex - 10))
        v = torch.where(b >= 128, -v, v)
    at = torch.arange(cols, device=q.device) // GROUP
    return v * _two(e.long() - 127)[:, at]


def _exact_rounded(x, kind):
    """The values that x (fp64) stands for after a checkpoint: the grid of each group, then the nearest point of it."""
    rows, cols = x.shape
    at = torch.arange(cols, device=x.device) // GROUP
    top = torch.zeros(rows, int(at[-1]) + 1, dtype=torch.float64, device=x.device)
    top.scatter_reduce_(1, at.expand(rows, cols), x.abs(), "amax")
    e = torch.ceil(torch.log2(top / TOP[kind])).clamp(min=-109)
    e = e - (top <= TOP[kind] * _two(e - 1)).double()  # log2 may be off next to a power of two
    e = (e + (top > TOP[kind] * _two(e)).double()).clamp(min=-110)
    unit = _two(e)[:, at]
    y = x / unit
    if kind == "int8":
        return torch.round(y) * unit
    step = _two(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)  # 3 bits after the first; 2^-9 at the bottom
    return torch.round(y / step) * step * unit


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "ckpt":
        return _exact_rounded(st["x"].double(), case["kind"])
    if case["op"] == "wgrad":
        out = []
        for dy, (q, e), s, g, g0 in zip(st["dy"], st["in"], st["scale"], st["g"], st["g0"]):
            p = torch.mm(dy.double().t().contiguous(), _exact_values(q, e, g.shape[1], case["kind"]))
            p = p if s is None else p * s.double()
            out.append(p if g0 is None else p + case["beta"] * g0.double())
        return out
    d = lambda k: None if st.get(k) is None else st[k].double()  # noqa: E731
    b, r, w1, w2, gate = d("b"), d("r"), d("w_pre"), d("w_post"), d("gate")
    a, c, post = st["res_scale"], st["branch_scale"], w2 is not None
    norm = lambda x: 1 / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS)  # noqa: E731
    one = torch.ones((), dtype=torch.float64, device=b.device)
    w2, gt = (w2 if post else one), (gate if gate is not None else one)
    out = {}
    if case["op"] == "bwd":
        u, v = (_exact_values(*st[k], case["cols"], case["kind"]) for k in ("u", "v"))
        ry, rb = st["rstd_y"].double()[:, None], st["rstd_b"].double()[:, None] if post else one
    else:
        rb = norm(b) if post else one
        y = a * r + c * gt * w2 * b * rb
        ry = norm(y)
        out = {"y": y, "h": y * ry * w1}
        if case["op"] == "fwd":
            return out
        u, v = _exact_rounded(y * ry, case["kind"]), _exact_rounded(b * rb, case["kind"])
    # y = a r + c gate n, n = w2 v, v = b / rms(b); h = w1 u, u = y / rms(y). Through a norm x -> x / rms(x) a
    # gradient d becomes (d - x^ <d, x^> / cols) / rms, x^ the normalised row.
    pull = lambda t, z, inv: inv * (t - z * ((t * z).sum(1, keepdim=True) / t.shape[1]))  # noqa: E731
    dh = d("dh")
    s = d("dy") + pull(dh * w1, u, ry)
    out["d_residual"] = a * s
    out["d_w_pre"] = torch.sum(dh * u, 0)
    dgate = c * s * w2 * v
    out["d_gate"] = None if gate is None else dgate if gate.dim() == 2 else torch.sum(dgate, 0)
    out["d_w_post"] = torch.sum(c * s * gt * v, 0) if post else None
    db = c * s * gt * w2
    out["d_branch"] = pull(db, v, rb) if post else db
    return out
