"""The 8-bit layer's operators as measured cases.

Every case has a plain form (elementary torch operations, 32 bits or more) and
the calls a user makes of ``sharded_state_amd``; ``own`` says which of the two
``run`` takes.  Kinds of cases:

  norm        h = x + residual, its root-mean-square norm, that in 8-bit blocks
  norm_grads  the norm's gradients, the residual path's added: dx and dw
  gather      a rank's master shard to 8-bit blocks, and the all-gather of the N ranks' blocks
              into the full buffer
  linear      y = x W^T with W in 8-bit blocks and x quantised on the way
  layer       the norm and the product that reads it
  grads       the gradients of that product: dx and dw, in the type of x as the reduce-scatter takes them

8-bit blocks: 128 elements of a row (of a 128 x 128 tile with ``tile``) share a power of two 2^e, e the
smallest whole number from -126 on with max|x| <= 448 * 2^e, and each is the e4m3 number nearest to
x / 2^e, ties to the even one, times 2^e.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def block_numel(d):
    """Elements of a GPT-2-style block: norms, qkv, projection and a 4d MLP, with biases."""
    return 12 * d * d + 13 * d


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token's residual stream in GPT-2 Large: latency
        dict(name="norm GPT-2 Large one token", kind="norm", m=1, d=1280, dtype="bf16", hdtype="bf16"),
        # a training step of the 70B shape with the residual stream in fp32, a ragged number of tokens
        dict(name="norm 70B fp32 stream", kind="norm", m=8191, d=8192, dtype="bf16", hdtype="f32"),
        # GPT-2 XL's backward, a ragged number of tokens
        dict(name="norm grads GPT-2 XL", kind="norm_grads", m=1000, d=1600, dtype="f16", hdtype="f16"),
        # the 70B shape's backward
        dict(name="norm grads 70B", kind="norm_grads", m=8192, d=8192, dtype="bf16", hdtype="bf16"),
        # GPT-2 XL's block on two ranks
        dict(name="gather GPT-2 XL N=2", kind="gather", numel=block_numel(1600), world=2, rank=0, dtype="f32",
             compute="f16"),
        # one 70B-shaped block on eight ranks
        dict(name="gather 70B N=8", kind="gather", numel=855638016, world=8, rank=7, dtype="f32", compute="bf16"),
        # one token through the 70B shape's gate
        dict(name="linear 70B one token", kind="linear", m=1, n=28672, k=8192, dtype="bf16", tile=False),
        # a prompt through the 13B shape's MLP
        dict(name="linear 13B prompt", kind="linear", m=4096, n=20480, k=5120, dtype="bf16", tile=False),
        # a batch of single tokens into GPT-2 XL's MLP, its weights in 128 x 128 tiles
        dict(name="layer GPT-2 XL 24 tokens", kind="layer", m=24, n=6400, k=1600, dtype="f16", tile=True),
        # a prompt into the 13B shape's qkv
        dict(name="layer 13B prompt", kind="layer", m=2000, n=15360, k=5120, dtype="bf16", tile=True),
        # a training step's backward through GPT-2 XL's MLP: a ragged number of tokens
        dict(name="grads GPT-2 XL", kind="grads", m=1000, n=6400, k=1600, dtype="f16", tile=False),
        # a training step's backward through the 70B shape's qkv
        dict(name="grads 70B", kind="grads", m=8192, n=10240, k=8192, dtype="bf16", tile=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_grads", "gather", "linear", "layer", "grads"])
    dt = rng.choice(["f16", "bf16", "f32"])
    if kind in ("norm", "norm_grads"):
        return dict(kind=kind, m=_log(rng, 1, 8192), d=_log(rng, 16, 16000), dtype=dt, hdtype=rng.choice([dt, "f32"]))
    if kind == "gather":
        world = rng.choice([1, 2, 3, 4, 8])
        return dict(kind=kind, numel=_log(rng, 1000, 200_000_000), world=world, rank=rng.randrange(world),
                    dtype=dt, compute=rng.choice(["f32", "f16", "bf16"]))
    m, n, k = _log(rng, 1, 4096), _log(rng, 64, 12000), _log(rng, 64, 9000)
    return dict(kind=kind, m=m, n=n, k=k, dtype=rng.choice(["f16", "bf16"]), tile=rng.random() < 0.5)


# ------------------------------------------------------------------ 8-bit blocks, plain
def _up(n):
    return -(-n // 128) * 128


def _padded(x, rows, cols):
    """x in 32 bits in a rows x cols matrix, zeros behind it."""
    if x.shape == (rows, cols):
        return x.float()
    out = torch.zeros((rows, cols), dtype=torch.float32, device=x.device)
    out[:x.shape[0], :x.shape[1]] = x
    return out


def _two(e):
    """2^e in 32 bits, for e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _exponents(a):
    """The blocks' e from their largest magnitudes in 32 bits."""
    bits = a.view(torch.int32)
    return ((bits >> 23) - 135 + ((bits & 0x7fffff) > 0x600000).int()).clamp(min=-126)


def _blocks(x, tile=False):
    """(codes [rows, cols up to 128] as e4m3, e [rows or rows / 128, blocks]) of finite x."""
    rows, cols = x.shape
    v = _padded(x, _up(rows) if tile else rows, _up(cols))
    g = v.view(-1, 128 if tile else 1, v.shape[1] // 128, 128)
    e = _exponents(g.abs().amax(dim=(1, 3)))
    q = (g * _two(-e)[:, None, :, None]).view(v.shape)[:rows]
    return q.to(torch.float8_e4m3fn), e


def _values(codes, e, cols):
    """The 32-bit values [rows, cols] of blocks."""
    rows = codes.shape[0]
    f = _two(e) if e.shape[0] == rows else _two(e).repeat_interleave(128, dim=0)[:rows]
    return (codes.float().view(rows, -1, 128) * f[:, :, None]).view(rows, -1)[:, :cols]


def _q32(x, tile=False):
    """x rounded to 8-bit blocks along its columns, in 32 bits."""
    return _values(*_blocks(x, tile), x.shape[1])


# ------------------------------------------------------------------ inputs
def _rand(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _kept(codes, e):
    """Blocks as a program holds them: bytes of codes and of scales."""
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _given(kept):
    return kept[0].view(torch.float8_e4m3fn), kept[1].int() - 127


def _layout(case):
    padded = -(-case["numel"] // case["world"]) * case["world"]
    return padded, padded // case["world"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, dt = case["kind"], DT[case["dtype"]]
    s = dict(case)
    if kind == "gather":
        padded, S = _layout(case)
        s["shard"] = _rand(g, (S,), 0.02, dt)
        s["peers"] = [None if q == case["rank"] else _kept(*_blocks(_rand(g, (1, S), 0.02, torch.float32)))
                      for q in range(case["world"])]
        s["full"] = torch.empty(padded, dtype=DT[case["compute"]], device="cuda")
        return s
    if kind in ("norm", "norm_grads", "layer"):
        # a stream whose rows differ in size, as they do between a model's first and last blocks
        d, hdt = case.get("d", case.get("k")), DT[case.get("hdtype", case["dtype"])]
        size = torch.exp(torch.randn((case["m"], 1), generator=g, device="cuda"))
        s["weight"] = (1 + _rand(g, (d,), 0.1, torch.float32)).to(dt)
        s["residual"] = (_rand(g, (case["m"], d), 2.0, torch.float32) * size).to(hdt)
        if kind == "norm_grads":
            s["h"] = s.pop("residual")
            s["rstd"] = (s["h"].double().square().mean(dim=1) + EPS).rsqrt().float()
            s["dy"] = _rand(g, (case["m"], d), 1e-2, dt)
            s["dh"] = _rand(g, (case["m"], d), 1e-2, hdt)
            return s
        s["x"] = _rand(g, (case["m"], d), 0.5, dt)
        if kind == "norm":
            return s
    m, n, k = case["m"], case["n"], case["k"]
    w = _rand(g, (n, k), 0.02, torch.float32)
    if kind != "layer":
        s["x"] = _rand(g, (m, k), 1.0, dt)
    if kind == "grads":
        s["dy"] = _rand(g, (m, n), 1e-2, dt)
        w = w.t().contiguous()
    s["w"] = _kept(*_blocks(w, case["tile"]))
    return s


# ------------------------------------------------------------------ plain forms
def _norm(s):
    h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    f = h.float()
    r = (f.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
    return h, r, f * r * s["weight"].float()


def _plain(s):
    kind = s["kind"]
    if kind == "norm":
        h, r, y = _norm(s)
        codes, e = _blocks(y)
        return dict(codes=codes, scales=(e + 127).to(torch.uint8).view(torch.float8_e8m0fnu), h=h, rstd=r[:, 0])
    if kind == "norm_grads":
        h, r, dy = s["h"].float(), s["rstd"][:, None], s["dy"].float()
        g = dy * s["weight"].float()
        dx = r * (g - h * (r * r * (g * h).mean(dim=1, keepdim=True))) + s["dh"].float()
        return dict(dx=dx.to(s["h"].dtype), dw=(dy * h * r).sum(dim=0))
    if kind == "gather":
        S = s["shard"].numel()
        mine = _q32(s["shard"].view(1, -1))[0]
        return s["full"].copy_(torch.cat([mine if p is None else _values(*_given(p), S)[0] for p in s["peers"]]))
    if kind == "linear":
        return (_q32(s["x"]) @ _values(*_given(s["w"]), s["k"]).t()).to(s["x"].dtype)
    if kind == "layer":
        h, r, y = _norm(s)
        return dict(h=h, y=(_q32(y) @ _values(*_given(s["w"]), s["k"]).t()).to(s["x"].dtype))
    dx = (_q32(s["dy"]) @ _values(*_given(s["w"]), s["n"]).t()).to(s["x"].dtype)
    return dict(dx=dx, dw=(_q32(s["dy"].t()) @ _q32(s["x"].t()).t()).to(s["x"].dtype))


# ------------------------------------------------------------------ the framework's calls
def _mine(s):
    import sharded_state_amd as ss
    kind = s["kind"]
    if kind == "norm":
        o = ss.fsdp_rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS)
        return dict(codes=o.q.codes.view(torch.float8_e4m3fn), scales=o.q.scales.view(torch.float8_e8m0fnu), h=o.h,
                    rstd=o.rstd)
    if kind == "norm_grads":
        dx, dw = ss.fsdp_rms_norm_grads(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"], dw_dtype=torch.float32)
        return dict(dx=dx, dw=dw)
    if kind == "gather":
        S = s["shard"].numel()
        mine = ss.fsdp_fp8_quantize(s["shard"])
        return ss.fsdp_fp8_gather([mine if p is None else ss.Fp8(p[0], p[1], S) for p in s["peers"]], s["full"])
    if kind == "linear":
        return ss.fsdp_fp8_linear(s["x"], ss.Fp8(*s["w"], s["k"], tile=s["tile"]))
    if kind == "layer":
        o = ss.fsdp_rms_norm_fp8(s["x"], s["weight"], s["residual"], eps=EPS)
        return dict(h=o.h, y=ss.fsdp_fp8_linear(o.q, ss.Fp8(*s["w"], s["k"], tile=s["tile"]), dtype=s["x"].dtype))
    dx, dw = ss.fsdp_fp8_linear_grads(s["dy"], s["x"], ss.Fp8(*s["w"], s["n"], tile=s["tile"]))
    return dict(dx=dx, dw=dw)


def run(state):
    return _mine(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    kind, b = case["kind"], SIZE[case["dtype"]]
    if kind in ("norm", "norm_grads"):
        m, d, hb = case["m"], case["d"], SIZE[case["hdtype"]]
        if kind == "norm":
            return dict(bytes=m * d * (b + 2 * hb + 129 / 128) + d * b + 4 * m, flops=8 * m * d)
        return dict(bytes=m * d * (b + 3 * hb) + d * (b + 4) + 4 * m, flops=12 * m * d)
    if kind == "gather":
        padded, S = _layout(case)
        return dict(bytes=S * b + padded * SIZE[case["compute"]] + (padded - S) * 129 / 128, flops=3 * S + padded)
    m, n, k = case["m"], case["n"], case["k"]
    w = n * k * (1 + 1 / (128 * 128 if case["tile"] else 128))
    if kind == "linear":
        return dict(bytes=m * k * b + w + m * n * b, flops=2 * m * n * k)
    if kind == "layer":
        return dict(bytes=3 * m * k * b + k * b + w + m * n * b, flops=2 * m * n * k + 8 * m * k)
    return dict(bytes=m * n * b + 2 * m * k * b + w + n * k * b, flops=4 * m * n * k)


# ------------------------------------------------------------------ 64 bits, from the definitions
def _power(e):
    """2^e in 64 bits of whole numbers e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _top_exponent(top):
    """The smallest e >= -126 with top <= 448 * 2^e, from top = f * 2^p with f in [1/2, 1): 448 = 0.875 * 2^9."""
    f, p = torch.frexp(top)
    return (p - 9 + (f > 0.875).to(p.dtype)).clamp(min=-126)


def _nearest(x, tile=False):
    """(code values, e) of x [rows, cols] along its columns in 64 bits: each number rounded to a whole number of
    its own steps, 1/8 of its binade and never under 2^-9.  In pieces, so that 64 bits fit."""
    rows, cols = x.shape
    high = 128 if tile else 1
    wide, blocks = _up(cols), _up(cols) // 128
    out = torch.empty(rows, wide, dtype=torch.float64, device=x.device)
    es = torch.empty(-(-rows // high), blocks, dtype=torch.int64, device=x.device)
    per = max(1, (1 << 25) // wide // high) * high
    for r in range(0, rows, per):
        for c in range(0, wide, 1 << 25):
            part = x[r:r + per, c:min(c + (1 << 25), cols)].double()
            n, w = part.shape
            v = torch.nn.functional.pad(part, (0, -w % 128, 0, -n % high))
            v = v.reshape(v.shape[0] // high, high, -1, 128)
            e = _top_exponent(v.abs().amax(dim=(1, 3)))
            y = v / _power(e)[:, None, :, None]
            step = _power((torch.frexp(y)[1] - 4).clamp(min=-9))
            y = (torch.round(y / step) * step).reshape(-1, v.shape[2] * 128)[:n]
            out[r:r + n, c:c + y.shape[1]] = y
            es[r // high:r // high + e.shape[0], c // 128:c // 128 + e.shape[1]] = e
    return out, es


def _times(codes, e, cols):
    """The 64-bit values of code values and exponents."""
    per = 1 if e.shape[0] == codes.shape[0] else 128
    f = _power(e).repeat_interleave(per, dim=0)[:codes.shape[0]].repeat_interleave(128, dim=1)
    return (codes * f)[:, :cols]


def _decoded(kept, cols):
    """The 64-bit values of bytes, from the fields of each code."""
    c = kept[0].to(torch.int64)
    exp, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(exp == 0, man * 2.0 ** -9, _power(exp - 7) * (1 + man / 8))
    return _times(torch.where(c >= 128, -mag, mag), kept[1].to(torch.int64) - 127, cols)


def _rounded(x, tile=False):
    return _times(*_nearest(x, tile), x.shape[1])


def _exact_norm(s):
    h = (s["x"].double() + s["residual"].double()).to(s["residual"].dtype).double()
    r = 1 / torch.sqrt((h ** 2).sum(dim=1, keepdim=True) / h.shape[1] + EPS)
    return h, r, h * r * s["weight"].double()


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        h, r, y = _exact_norm(s)
        codes, e = _nearest(y)
        return dict(codes=codes, scales=_power(e), h=h, rstd=r[:, 0])
    if kind == "norm_grads":
        h, w, dy = s["h"].double(), s["weight"].double(), s["dy"].double()
        r = s["rstd"].double()[:, None]
        n = h * r                                       # the normed rows, before the weight
        back = dy * w - n * ((dy * w * n).sum(dim=1, keepdim=True) / h.shape[1])
        return dict(dx=r * back + s["dh"].double(), dw=(dy * n).sum(dim=0))
    if kind == "gather":
        S = s["shard"].numel()
        full = torch.empty(s["full"].numel(), dtype=torch.float64, device="cuda")
        for q, p in enumerate(s["peers"]):
            at = full[q * S:(q + 1) * S]
            for c in range(0, S, 1 << 24):
                e = min(S, c + (1 << 24))
                if p is None:
                    at[c:e] = _rounded(s["shard"][c:e].view(1, -1))[0]
                else:
                    at[c:e] = _decoded((p[0][:, c:_up(e)], p[1][:, c // 128:_up(e) // 128]), e - c)[0]
        return full
    if kind == "linear":
        return _rounded(s["x"]) @ _decoded(s["w"], case["k"]).t()
    if kind == "layer":
        h, r, y = _exact_norm(s)
        return dict(h=h, y=_rounded(y) @ _decoded(s["w"], case["k"]).t())
    dx = _rounded(s["dy"]) @ _decoded(s["w"], case["n"]).t()
    return dict(dx=dx, dw=_rounded(s["dy"].t().contiguous()) @ _rounded(s["x"].t().contiguous()).t())
