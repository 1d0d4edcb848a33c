"""The block-boundary, int8 and gradient-clipping operators: cases, inputs, plain forms and exact values.

Three operators of the library, each in its plain form (elementary torch operations in
32 bits, 64 where 32 lose what matters) and through its public call:

- boundary (forward and backward): between two blocks, the branch output o is normalised by
  group, gated by u, scaled and added to the residual stream x, and the next block's GroupLN
  reads the sum:  h = x + s_g (GLN_post(o) f(u)),  y = GLN_pre(h);
- linear_i8: activations (float rows, quantised per token within the call, or int8 rows with
  their scales) times int8 weights with a scale per output channel, with the block's epilogues;
- clip: the global 2-norm over many gradient tensors, the loss scale taken out, and clipping.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
NORM_EPS = 1e-6
TINY = 2.0 ** -100  # smallest row maximum a quantised row's scale is taken from
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}
GROUP_SCALE = (1.0, 3.0, 0.3, 10.0)  # U, S, R, C token features


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one request's few candidates between two blocks, as int8 rows for the next projection
        dict(name="boundary 8 candidates int8", op="boundary", T=8, d=512, branch="bf16", stream="f32", y="i8",
             gate="linear", post=True, scale=True, rows="candidates"),
        # the packed batch of the 512-wide block between two blocks
        dict(name="boundary block 512", op="boundary", T=200003, d=512, branch="bf16", stream="f32", y="bf16",
             gate="linear", post=True, scale=True, rows="users"),
        # the 1024-wide stack, its next projection in int8
        dict(name="boundary stack 1024 int8", op="boundary", T=65537, d=1024, branch="f16", stream="f32", y="i8",
             gate="silu", post=True, scale=True, rows="users"),
        # a small training batch, everything in fp32
        dict(name="boundary back 256 f32", op="boundary_back", T=1917, d=256, branch="f32", stream="f32", y="f32",
             gate="silu", post=True, scale=True, rows="users"),
        # the training step of the 512-wide block
        dict(name="boundary back 512", op="boundary_back", T=200003, d=512, branch="bf16", stream="f32", y="bf16",
             gate="linear", post=True, scale=True, rows="users"),
        # a chunk of eight candidates through the Q|K|V|U projection, quantised on the way
        dict(name="linear 8 rows", op="linear", M=8, N=2048, K=512, x="bf16", epi="none", out="f16", bias=False),
        # a chunk of candidates through MLP1 of the 1024-wide block
        dict(name="linear 1000 rows silu", op="linear", M=1000, N=4096, K=1024, x="bf16", epi="silu", out="bf16", bias=True),
        # Q|K|V|U projection of a whole batch from the int8 rows that a boundary left
        dict(name="linear block 512", op="linear", M=131075, N=2048, K=512, x="i8", epi="none", out="f16", bias=False),
        # MLP2 of the 1024-wide block with its residual, its hidden rows quantised on the way
        dict(name="linear mlp2 1024", op="linear", M=65543, N=1024, K=4096, x="bf16", epi="resid", out="f32", bias=True),
        # one 512-wide block's gradients, biases among them
        dict(name="clip block 512", op="clip", L=1, d=512, ff=2048, kind="f32", to="f32", bias=True, odd=0),
        # an eight-block stack's gradients
        dict(name="clip stack 1024", op="clip", L=8, d=1024, ff=4096, kind="f32", to="f32", bias=False, odd=0),
        # many small vectors of odd sizes beside a small block with bf16 weight gradients
        dict(name="clip odd tensors", op="clip", L=1, d=64, ff=256, kind="bf16", to="bf16", bias=True, odd=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["boundary", "boundary_back", "linear", "linear", "clip"])
    if op in ("boundary", "boundary_back"):
        d = 8 * _log(rng, 8, 256)
        stream = rng.choice(["f32", "f32", "bf16"])
        y = rng.choice(["bf16", "f32", "i8"] if op == "boundary" else ["bf16", "f32"])
        most = 100_000_000 // d if op == "boundary" else 60_000_000 // d
        return dict(op=op, T=_log(rng, 1, most), d=d, branch=rng.choice(["bf16", "f16", "f32"]), stream=stream, y=y,
                    gate=rng.choice(["none", "linear", "silu"]), post=rng.random() < 0.8, scale=rng.random() < 0.8,
                    rows=rng.choice(["users", "candidates"]))
    if op == "linear":
        N, K = 8 * _log(rng, 8, 512), 16 * _log(rng, 4, 256)
        most = min(131072, int(2.7e11 / (N * K)), int(2.6e8 / (N + K)))
        epi, x = rng.choice(["none", "silu", "resid"]), rng.choice(["bf16", "f32", "i8"])
        return dict(op=op, M=_log(rng, 1, most), N=N, K=K, x=x, epi=epi,
                    out="f32" if epi == "resid" else rng.choice(["bf16", "f16", "f32"]), bias=rng.random() < 0.5)
    d = 64 * _log(rng, 1, 14)
    # f16 gradients leave as fp32: with the loss scale taken out they would be f16 subnormals
    kind, to = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
    return dict(op=op, L=rng.randint(1, 6), d=d, ff=64 * _log(rng, 1, 64), kind=kind, to=to,
                bias=rng.random() < 0.3, odd=rng.randint(0, 3))


def clip_shapes(c):
    """Shapes of the gradients of L blocks (per-group norms, projections, MLP), then `odd` small odd vectors."""
    d, ff = c["d"], c["ff"]
    block = [(4, d), (4, d), (4 * d, d), (4, d), (4, d), (ff, d), (d, ff)]
    if c["bias"]:
        block += [(4 * d,), (ff,), (d,)]
    return block * c["L"] + [(1 + (i * i * 37 + 11 * i) % 1999,) for i in range(c["odd"])]


def outputs_of(c):
    """Names of a boundary's outputs."""
    if c["op"] == "boundary":
        return ["h", "y"] + (["y_scale"] if c["y"] == "i8" else [])
    names = ["dx", "do"] + (["du"] if c["gate"] != "none" else []) + ["pre_gamma", "pre_beta"]
    return names + (["post_gamma", "post_beta"] if c["post"] else []) + (["scale"] if c["scale"] else [])


# ----------------------------------------------------------------- inputs --
def _groups(c, seed):
    """Group ids of the packed rows: whole users (U, S, R, C segments), or candidates alone."""
    T = c["T"]
    if c["rows"] == "candidates":
        return torch.full((T,), 3, dtype=torch.int8, device="cuda")
    rng = np.random.default_rng(seed)
    n = T // 300 + 1  # a user has 24 + at least 300 tokens
    lens = np.stack([np.full(n, 24), rng.integers(300, 1001, n), rng.integers(20, 101, n), rng.integers(32, 257, n)], 1)
    ids = np.repeat(np.tile(np.arange(4, dtype=np.int8), n), lens.reshape(-1))[:T]
    return torch.from_numpy(ids).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(shift).to(dtype)

    if c["op"] in ("boundary", "boundary_back"):
        T, d, bt, st = c["T"], c["d"], TYPES[c["branch"]], TYPES[c["stream"]]
        gid = _groups(c, seed)
        feature = torch.tensor(GROUP_SCALE, device="cuda")[gid.long()][:, None]
        s = dict(case=c, group_id=gid, o=normal(T, d, dtype=bt, shift=0.1), x=(normal(T, d) * feature).to(st), u=None)
        if c["gate"] != "none":  # the gate is the last quarter of the Q|K|V|U rows
            s["u"] = normal(T, 4 * d, dtype=bt, scale=0.7)[:, 3 * d:]
        one = lambda shift, scale: normal(4, d, shift=shift, scale=scale)  # noqa: E731
        s["post_gamma"], s["post_beta"] = (one(1.0, 0.3), one(0.0, 0.3)) if c["post"] else (None, None)
        s["scale"] = one(0.5, 0.1) if c["scale"] else None
        s["pre_gamma"], s["pre_beta"] = one(1.0, 0.3), one(0.0, 0.3)
        if c["op"] == "boundary_back":
            s["dh"] = normal(T, d, dtype=st, scale=0.01)
            s["dy"] = normal(T, d, dtype=TYPES[c["y"]], scale=0.01)
        return s
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        s = dict(case=c, bias=normal(N) if c["bias"] else None, resid=normal(M, N, scale=2.0) if c["epi"] == "resid" else None)
        s["w"] = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        s["w_scale"] = normal(N, scale=0.1, shift=1.0).abs_().clamp_(min=0.1).mul_(1.0 / (73.0 * math.sqrt(K)))
        if c["x"] == "i8":
            s["x"] = normal(M, K, scale=32.0).round_().clamp_(-127, 127).to(torch.int8)
            s["x_scale"] = normal(M).abs_().add_(0.5).mul_(1.0 / 32.0)
        else:
            x = normal(M, K)
            x *= torch.rand(K, generator=g, device="cuda").mul_(4.0).square_().add_(0.1)  # some channels much larger than others
            if M > 4:
                x[M // 2] = 0.0  # a padding row
            s["x"], s["x_scale"] = x.to(TYPES[c["x"]]), None
        return s
    shapes, t = clip_shapes(c), TYPES[c["kind"]]
    grads = [normal(*sh, dtype=t if len(sh) == 2 else torch.float32, scale=0.02 * (1 + i % 3)) for i, sh in enumerate(shapes)]
    s = dict(case=c, grads=grads, inv_scale=1.0 / 1024.0)
    s["max_norm"] = 1e-3 * math.sqrt(sum(x.numel() for x in grads)) * s["inv_scale"]  # well below the norm: it clips
    s["types"] = [TYPES[c["to"]] if len(sh) == 2 else torch.float32 for sh in shapes]
    if own:
        import generative_recommendation_ranking_b200 as mt

        s["outs"] = [torch.empty_like(x, dtype=to) for x, to in zip(grads, s["types"])]
        s["set"] = mt.GradientSet(grads, s["outs"])
    return s


# ------------------------------------------------------------- plain forms --
def _norm(v, gamma, beta):
    """(normalised rows, output, 1 / sigma) of GroupLN in fp32; gamma and beta per row."""
    c = v - v.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    return c * rstd, c * rstd * gamma + beta, rstd


def _quantise(y):
    scale = y.abs().amax(1).float().clamp(min=TINY) / 127.0
    # the quotient in 64 bits: a value next to a border goes where it belongs
    return torch.round(y.double() / scale.double()[:, None]).clamp_(-127, 127), scale


def _boundary_plain(s):
    c, gid = s["case"], s["group_id"].long()
    o, x = s["o"].float(), s["x"].float()
    ohat = rstd_o = None
    n = o
    if c["post"]:
        ohat, n, rstd_o = _norm(o, s["post_gamma"][gid], s["post_beta"][gid])
    f = None
    if c["gate"] != "none":
        u = s["u"].float()
        f = u if c["gate"] == "linear" else u / (1.0 + torch.exp(-u))
    p = n if f is None else n * f
    scale = s["scale"][gid] if c["scale"] else 1.0
    h = x + p * scale
    hhat, y, rstd_h = _norm(h, s["pre_gamma"][gid], s["pre_beta"][gid])
    if c["op"] == "boundary":
        if c["y"] != "i8":
            return dict(h=h.to(s["x"].dtype), y=y.to(TYPES[c["y"]]))
        q, ys = _quantise(y)
        return dict(h=h.to(s["x"].dtype), y=(q * ys[:, None]).to(torch.bfloat16), y_scale=ys)
    # by group over the rows, in 64 bits: long sums
    pick = (gid[None, :] == torch.arange(4, device="cuda")[:, None]).double()
    per_group = lambda v: (pick @ v.double()).float()  # noqa: E731
    dy = s["dy"].float()
    out = dict(pre_gamma=per_group(dy * hhat), pre_beta=per_group(dy))
    a = dy * s["pre_gamma"][gid]
    dh = s["dh"].float() + rstd_h * (a - a.mean(1, keepdim=True) - hhat * (a * hhat).mean(1, keepdim=True))
    out["dx"] = dh.to(s["x"].dtype)
    if c["scale"]:
        out["scale"] = per_group(dh * p)
    dp = dh * scale
    dn = dp
    if f is not None:
        dn, df = dp * f, dp * n
        if c["gate"] == "silu":
            sig = 1.0 / (1.0 + torch.exp(-u))
            df = df * sig * (1.0 + u * (1.0 - sig))
        out["du"] = df.to(s["o"].dtype)
    do = dn
    if c["post"]:
        out["post_gamma"], out["post_beta"] = per_group(dn * ohat), per_group(dn)
        b = dn * s["post_gamma"][gid]
        do = rstd_o * (b - b.mean(1, keepdim=True) - ohat * (b * ohat).mean(1, keepdim=True))
    out["do"] = do.to(s["o"].dtype)
    return out


def _linear_plain(s):
    c = s["case"]
    q, xs = (s["x"], s["x_scale"]) if c["x"] == "i8" else _quantise(s["x"])
    v = (q.float() @ s["w"].float().T) * xs[:, None] * s["w_scale"]
    if c["bias"]:
        v = v + s["bias"]
    if c["epi"] == "silu":
        v = v / (1.0 + torch.exp(-v))
    elif c["epi"] == "resid":
        v = v + s["resid"]
    return v.to(TYPES[c["out"]])


def _clip_plain(s):
    # the sum over all tensors in 64 bits: a long sum
    norm = torch.stack([x.double().square().sum() for x in s["grads"]]).sum().sqrt().float() * s["inv_scale"]
    coef = s["inv_scale"] * (s["max_norm"] / (norm + NORM_EPS)).clamp(max=1.0)
    return dict(norm=norm.reshape(1), grads=[(x.float() * coef).to(to) for x, to in zip(s["grads"], s["types"])])


# --------------------------------------------------------- the own calls --
def _own(s):
    import generative_recommendation_ranking_b200 as mt

    c = s["case"]
    if c["op"] == "boundary":
        h, y, ys = mt.boundary_forward(s["x"], s["o"], s["u"], s["group_id"], s["post_gamma"], s["post_beta"], s["scale"],
                                       s["pre_gamma"], s["pre_beta"], gate=c["gate"], y_dtype=TYPES[c["y"]])
        if c["y"] != "i8":
            return dict(h=h, y=y)
        value = torch.empty(y.shape, dtype=torch.bfloat16, device=y.device)  # what the int8 rows stand for
        return dict(h=h, y=torch.mul(y, ys[:, None], out=value), y_scale=ys)
    if c["op"] == "boundary_back":
        return mt.boundary_backward(s["x"], s["o"], s["u"], s["group_id"], s["post_gamma"], s["post_beta"], s["scale"],
                                    s["pre_gamma"], s["pre_beta"], s["dh"], s["dy"], gate=c["gate"])
    if c["op"] == "linear":
        epi = {"none": mt.MTGR_EPI_NONE, "silu": mt.MTGR_EPI_SILU, "resid": mt.MTGR_EPI_RESID}[c["epi"]]
        return mt.linear_i8(s["x"], s["w"], s["w_scale"], x_scale=s["x_scale"], bias=s["bias"], epi=epi, resid=s["resid"],
                            out_dtype=TYPES[c["out"]])
    norm = s["set"].clip(s["max_norm"], s["inv_scale"])
    return dict(norm=norm, grads=s["outs"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _linear_plain(state) if op == "linear" else _clip_plain(state) if op == "clip" else _boundary_plain(state)


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["op"] in ("boundary", "boundary_back"):
        n, b, st, y = c["T"] * c["d"], SIZE[c["branch"]], SIZE[c["stream"]], SIZE[c["y"]]
        gate = c["gate"] != "none"
        small = c["T"] + 4 * c["d"] * 4 * (2 + 2 * c["post"] + c["scale"])
        if c["op"] == "boundary":  # o, u, x in; h, y out
            return dict(bytes=n * (b * (1 + gate) + 2 * st + y) + small + (4 * c["T"] if y == 1 else 0), flops=20 * n)
        return dict(bytes=n * (2 * b * (1 + gate) + 3 * st + y) + 2 * small, flops=50 * n)
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        moved = M * K * SIZE[c["x"]] + N * K + M * N * SIZE[c["out"]] + 4 * N * (1 + c["bias"])
        moved += 4 * M * N if c["epi"] == "resid" else 0
        return dict(bytes=moved + (4 * M if c["x"] == "i8" else 0), flops=2 * M * N * K)
    sizes = [(math.prod(sh), SIZE[c["kind"]] + SIZE[c["to"]] if len(sh) == 2 else 8) for sh in clip_shapes(c)]
    return dict(bytes=sum(n * b for n, b in sizes), flops=3 * sum(n for n, _ in sizes))


# ------------------------------------------------------------ exact values --
def exact(case, seed):
    """The outputs from the definitions in 64 bits: the backward by differentiating the forward."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "clip":
        flat = torch.cat([x.reshape(-1).double() for x in s["grads"]])
        norm = torch.linalg.vector_norm(flat) * s["inv_scale"]
        coef = s["inv_scale"] * min(1.0, s["max_norm"] / (float(norm) + NORM_EPS))
        return dict(norm=norm.reshape(1), grads=[x.double() * coef for x in s["grads"]])
    if c["op"] == "linear":
        x = s["x"].double()
        if c["x"] == "i8":
            xs = s["x_scale"].double()
        else:
            xs = (s["x"].float().abs().max(dim=1).values.clamp(min=TINY) / 127.0).double()  # a scale is a 32-bit number
            x = torch.round(x / xs.unsqueeze(1))
        v = torch.einsum("mk,nk->mn", x * xs.unsqueeze(1), s["w"].double() * s["w_scale"].double().unsqueeze(1))
        if c["bias"]:
            v += s["bias"].double()
        return torch.nn.functional.silu(v) if c["epi"] == "silu" else v + s["resid"].double() if c["epi"] == "resid" else v
    back = c["op"] == "boundary_back"
    rows = s["group_id"].long()
    leaf = {k: s[k].double().requires_grad_(back) for k in ("x", "o", "u", "post_gamma", "post_beta", "scale", "pre_gamma",
                                                             "pre_beta") if s[k] is not None}

    def group_norm(v, which):
        z = torch.nn.functional.layer_norm(v, (c["d"],), eps=EPS)
        return torch.addcmul(leaf[which + "_beta"].index_select(0, rows), z, leaf[which + "_gamma"].index_select(0, rows))

    with torch.set_grad_enabled(back):
        branch = group_norm(leaf["o"], "post") if c["post"] else leaf["o"]
        if c["gate"] != "none":
            branch = branch * (leaf["u"] if c["gate"] == "linear" else torch.nn.functional.silu(leaf["u"]))
        if c["scale"]:
            branch = branch * leaf["scale"].index_select(0, rows)
        h = leaf["x"] + branch
        y = group_norm(h, "pre")
    if not back:
        out = dict(h=h, y=y)
        if c["y"] == "i8":
            out["y_scale"] = y.abs().max(dim=1).values.clamp(min=TINY) / 127.0
            step = out["y_scale"].float().double().unsqueeze(1)
            out["y"] = torch.round(y / step) * step
        return out
    torch.autograd.backward([h, y], [s["dh"].double(), s["dy"].double()])
    names = {"dx": "x", "do": "o", "du": "u"}
    return {k: leaf[names.get(k, k)].grad for k in outputs_of(c)}
