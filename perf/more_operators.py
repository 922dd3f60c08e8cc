"""What the residual norm, the 8-bit integer product and the layer for a few tokens are measured
on: the cases, their inputs, a plain form of each operator in elementary torch operations, and
each operator's value in 64 bits.

Operators (the case's "op"):

norm      rows x and a residual -> their sum, and the sum's root-mean-square norm times a
          weight: r = x + residual, rounded to the residual's type (without one, r = x);
          p = r w; rstd = 1 / sqrt(mean(r^2) + eps); the values are p rstd.  They come out
          in the type of x, or as codes: e4m3 with one scale for each block of 128 along the row
          (code of 448 p / a, scale a rstd / 448, a the block's largest |p|), or int8 with one
          scale for the row (code 127 p / a to the nearest integer, scale a rstd / 127).
quantize  rows -> int8 codes with one fp32 scale each: a the row's largest magnitude, the scale
          a / 127 and the code of x the integer nearest to 127 x / a (halves to even).
gemm      y = x W^T on int8 codes, x with a scale for each row, W with one for each output.
token     the whole MoE layer for a few tokens: softmax top-k router, gate/up, SwiGLU, down,
          weighted sum, shared expert; on bf16 weights or on e4m3 ones with a scale for each
          128 x 128 block.  "given": the experts and weights of the rows come from outside.

Each call writes its outputs to buffers that the caller keeps.  The inputs of a case are made
from its seed alone.  int8 codes are whole numbers and compared as such.
"""
from __future__ import annotations

import torch

own = False   # False: the plain forms; True: the library's calls

FP8_MAX = 448.0      # the largest e4m3 value
I8_MAX = 127.0
BLOCK = 128
AMAX_MIN = 2.0 ** -100   # a block's (or row's) largest magnitude counts as at least this
EPS = 1e-6


# ---------------------------------------------------------------------------- cases

def _norm(R, H, dtype, residual, out, weight, pad=0):
    return {"op": "norm", "R": R, "H": H, "dtype": dtype, "residual": residual, "out": out,
            "weight": weight, "pad": pad}


def _token(R, codes, given=False, H=2048, E=256, k=8, I=512, Is=512):
    return {"op": "token", "R": R, "codes": codes, "given": given, "H": H, "E": E, "k": k, "I": I, "Is": Is}


def listed():
    return [
        # the norm before a layer, one token of a decoding step
        {"name": "norm-1", **_norm(1, 2048, "bf16", "bf16", "same", "bf16")},
        # a ragged batch of an odd width, rows of a wider buffer, an fp32 residual stream, codes
        # for the integer product
        {"name": "norm-777-odd", **_norm(777, 1000, "f16", "f32", "i8", "f32", 24)},
        # a prompt of 8192 tokens, codes for the e4m3 product
        {"name": "norm-8192", **_norm(8192, 2048, "bf16", "bf16", "e4m3", "bf16")},
        # the rows of one denoising pass over a block, and a prompt's
        {"name": "quantize-32", "op": "quantize", "R": 32, "K": 2048, "dtype": "bf16"},
        {"name": "quantize-8192", "op": "quantize", "R": 8192, "K": 2048, "dtype": "bf16"},
        # one token through a projection of the layer's width
        {"name": "gemm-1", "op": "gemm", "R": 1, "N": 2048, "K": 2048, "out": "bf16"},
        # ragged in every direction
        {"name": "gemm-77-odd", "op": "gemm", "R": 77, "N": 1000, "K": 1104, "out": "f32"},
        # a prompt through a projection to twice the layer's width
        {"name": "gemm-8192", "op": "gemm", "R": 8192, "N": 4096, "K": 2048, "out": "bf16"},
        # one token of a decoding step through the layer, in both weight types
        {"name": "token-1", **_token(1, "bf16")},
        {"name": "token-1-e4m3", **_token(1, "e4m3")},
        # three sequences decoded together on a small layer whose sizes end inside a block, their
        # routing made by a rule outside
        {"name": "token-3-odd", **_token(3, "e4m3", True, 1280, 64, 6, 320, 640)},
        # a denoising block of eight rows (or eight sequences)
        {"name": "token-8", **_token(8, "bf16")},
    ]


def _log_int(rng, lo, hi, of=1):
    """A multiple of `of`, evenly spread over the logarithm of lo .. hi (times `of`)."""
    return of * max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "quantize", "gemm", "token"])
    if op == "token":
        E = _log_int(rng, 8, 256)
        H, E, k, I, Is = rng.choice([(2048, 256, 8, 512, 512)] + 3 * [(
            256 * rng.randint(1, 8), E, rng.randint(1, 8), 64 * rng.randint(1, 8), 64 * rng.randint(1, 10))])
        return _token(rng.randint(1, 8), rng.choice(["bf16", "e4m3"]), rng.random() < 0.3, H, E, k, I, Is)
    R = _log_int(rng, 1, 8192)
    if op == "norm":
        H = _log_int(rng, 33, 4096)
        if rng.random() < 0.6:
            H = -(-H // 8) * 8
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return _norm(R, H, dtype, rng.choice(["none", dtype, dtype, "f32"]),
                     rng.choice(["same", "e4m3", "i8"]), rng.choice([dtype, dtype, "f32"]),
                     rng.choice([0, 0, 8, 3]))
    if op == "quantize":
        return {"op": op, "R": R, "K": _log_int(rng, 8, 255, of=rng.choice([1, 2, 8, 16])),
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    return {"op": op, "R": R, "N": _log_int(rng, 33, 4096), "K": _log_int(rng, 4, 128, of=16),
            "out": rng.choice(["bf16", "f16", "f32"])}


# --------------------------------------------------------------------------- inputs

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _e4m3_codes(p, a):
    """Codes of p with the largest magnitude a (broadcast): 448 p / a is formed as
    (7/8 p) / (a / 512), so that one rounding precedes the code's."""
    return (p * 0.875 / (a * 2.0 ** -9)).to(torch.float8_e4m3fn)


def _i8_codes(p, a):
    """Likewise 127 p / a as (127/128 p) / (a / 128), to the nearest integer."""
    return (p * (127.0 / 128.0) / (a * 2.0 ** -7)).round().to(torch.int8)


def _over(a, m):
    """a / m.  (a / m with a plain number m is formed as a product.)"""
    return a / torch.full_like(a, m)


def _block_codes(w):
    """Weights [..., N, K] -> e4m3 codes and fp32 scales [..., ceil(N/128), ceil(K/128)]."""
    *lead, N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    p = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N))
    p = p.view(*lead, nb, BLOCK, kb, BLOCK)
    a = p.abs().amax(dim=(-3, -1), keepdim=True).clamp_min(AMAX_MIN)
    q = _e4m3_codes(p, a).view(*lead, nb * BLOCK, kb * BLOCK)[..., :N, :K]
    return q.contiguous(), _over(a, FP8_MAX).reshape(*lead, nb, kb).contiguous()


def _rows_i8(x):
    """Rows -> int8 codes and their scales [R]."""
    x = x.float()
    a = x.abs().amax(1, keepdim=True).clamp_min(AMAX_MIN)
    return _i8_codes(x, a), _over(a, I8_MAX)[:, 0]


def _weights(g, lead, N, K, codes, sigma=0.02):
    """Seeded normal weights in bf16 (scales: None) or as block codes, a few matrices at a time."""
    n = 1
    for d in lead:
        n *= d
    qs, ss = [], []
    step = max(1, (1 << 27) // (N * K))
    for i in range(0, n, step):
        w = torch.randn(min(step, n - i), N, K, generator=g, device="cuda") * sigma
        if codes == "e4m3":
            q, s = _block_codes(w)
            ss.append(s)
        else:
            q = w.to(torch.bfloat16)
        qs.append(q)
    q = torch.cat(qs).view(*lead, N, K)
    return q, torch.cat(ss).view(*lead, *ss[0].shape[1:]) if ss else None


_WEIGHTS = ("wg", "wu", "wd", "sg", "su", "sd")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(1_000_003 * seed + 29)
    s = {"case": c}
    R = c["R"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if c["op"] == "norm":
        H, dt = c["H"], _DTYPES[c["dtype"]]
        wide = randn(R, H + c["pad"]) * torch.exp(0.5 * randn(R, 1))   # rows of unlike size
        s["x"] = wide.to(dt)[:, :H]
        s["w"] = (1.0 + 0.1 * randn(H)).to(_DTYPES[c["weight"]])
        if c["residual"] != "none":
            rt = _DTYPES[c["residual"]]
            s["res"] = (3.0 * randn(R, H)).to(rt)   # a stream that many layers have added to
            s["sum"] = torch.empty(R, H, dtype=rt, device="cuda")
        if c["out"] == "same":
            s["y"] = torch.empty(R, H, dtype=dt, device="cuda")
        elif c["out"] == "e4m3":
            s["codes"] = torch.empty(R, H, dtype=torch.float8_e4m3fn, device="cuda")
            s["scales"] = torch.empty(-(-H // BLOCK), R, device="cuda")
        else:
            s["codes"] = torch.empty(R, H, dtype=torch.int8, device="cuda")
            s["scales"] = torch.empty(R, device="cuda")
    elif c["op"] == "quantize":
        K = c["K"]
        s["x"] = (randn(R, K) * torch.exp(randn(R, 1))).to(_DTYPES[c["dtype"]])
        s["codes"] = torch.empty(R, K, dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(R, device="cuda")
    elif c["op"] == "gemm":
        N, K = c["N"], c["K"]
        s["xq"], s["xs"] = (t.contiguous() for t in _rows_i8(randn(R, K)))
        s["wq"], s["ws"] = (t.contiguous() for t in _rows_i8(0.02 * randn(N, K)))
        s["y"] = torch.empty(R, N, dtype=_DTYPES[c["out"]], device="cuda")
    else:
        H, E, k, I, Is = (c[n] for n in ("H", "E", "k", "I", "Is"))
        shapes = (((E,), I, H), ((E,), I, H), ((E,), H, I), ((), Is, H), ((), Is, H), ((), H, Is))
        for n, shape in zip(_WEIGHTS, shapes):
            s[n], s[n + "s"] = _weights(g, *shape, c["codes"])
        s["router"] = (0.02 * randn(E, H)).to(torch.bfloat16)
        s["x"] = randn(R, H).to(torch.bfloat16)
        if c["given"]:   # distinct experts per row, weights that sum to 1
            s["idx"] = randn(R, E).argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
            s["w"] = torch.softmax(randn(R, k), dim=1)
        else:
            s["idx"] = torch.empty(R, k, dtype=torch.int32, device="cuda")
            s["w"] = torch.empty(R, k, device="cuda")
        s["y"] = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    if own:   # what a program that calls the library keeps: its workspace, its layer
        from sparse_moe_layer_row_gb300 import moe_block as mb
        if c["op"] == "gemm":
            s["ws_mem"] = torch.zeros(mb.moe_i8_gemm_workspace_bytes(R, c["N"], c["K"]),
                                      dtype=torch.uint8, device="cuda")
        elif c["op"] == "token":
            w = [s[n] for n in _WEIGHTS]
            if c["codes"] == "e4m3":
                sc = [s[n + "s"] for n in _WEIGHTS]
                q = mb.Fp8Experts(*w[:3], *sc[:3], *w[3:], *sc[3:])
                s["layer"] = mb.MoeBlockLayer.fp8(s["router"], q, k=k, max_rows=R, max_blocks=1)
            else:
                s["layer"] = mb.MoeBlockLayer(s["router"], *w, k=k, max_rows=R, max_blocks=1)
    return s


# ----------------------------------------------------------------------- plain forms

def _plain_norm(s):
    c = s["case"]
    r = s["x"].float()
    out = []
    if c["residual"] != "none":
        total = (r + s["res"].float()).to(s["res"].dtype)
        out.append(total)
        r = total.float()
    p = r * s["w"].float()
    rstd = (1.0 / torch.sqrt(r.double().square().mean(1, keepdim=True) + EPS)).float()
    R, H = r.shape
    if c["out"] == "same":
        return out + [(p * rstd).to(s["x"].dtype)]
    if c["out"] == "i8":
        a = p.abs().amax(1, keepdim=True).clamp_min(AMAX_MIN)
        return out + [_i8_codes(p, a), _over(a * rstd, I8_MAX)[:, 0]]
    kb = -(-H // BLOCK)
    p = torch.nn.functional.pad(p, (0, kb * BLOCK - H)).view(R, kb, BLOCK)
    a = p.abs().amax(2, keepdim=True).clamp_min(AMAX_MIN)
    q = _e4m3_codes(p, a).view(R, kb * BLOCK)[:, :H].contiguous()
    return out + [q, _over(a[..., 0] * rstd, FP8_MAX).t().contiguous()]


def _rows_e4m3(x):
    """Rows -> their values after the rounding to e4m3 with a scale per block of 128, in fp32."""
    R, K = x.shape
    kb = -(-K // BLOCK)
    p = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(R, kb, BLOCK)
    a = p.abs().amax(2, keepdim=True).clamp_min(AMAX_MIN)
    return (_e4m3_codes(p, a).float() * _over(a, FP8_MAX)).view(R, kb * BLOCK)[:, :K]


def _values(q, sc):
    """Weights (bf16), or codes [..., N, K] and scales, in fp32."""
    if sc is None:
        return q.float()
    N, K = q.shape[-2:]
    return q.float() * sc.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]


def _plain_ffn(x, wg, wu, wd, codes):
    """x [T, n, H] through weights [T, ., .]."""
    g = torch.bmm(x, wg.transpose(1, 2))
    u = torch.bmm(x, wu.transpose(1, 2))
    h = g / (1.0 + torch.exp(-g)) * u
    if codes == "e4m3":
        h = _rows_e4m3(h.view(-1, h.shape[-1])).view(h.shape)
    return torch.bmm(h, wd.transpose(1, 2))


def _plain_token(s):
    c = s["case"]
    R, H, k = c["R"], c["H"], c["k"]
    idx, w = s["idx"], s["w"]
    if not c["given"]:
        z = s["x"].double() @ s["router"].double().t()   # 64 bits: the order of nearly equal logits
        top = z.sort(dim=1, descending=True, stable=True)
        idx = top.indices[:, :k].to(torch.int32)
        a = torch.exp(top.values[:, :k] - top.values[:, :1])
        w = (a / a.sum(1, keepdim=True)).float()
    x = s["x"].float()
    if c["codes"] == "e4m3":
        x = _rows_e4m3(x)

    def take(n, at):
        return _values(s[n][at], None if s[n + "s"] is None else s[n + "s"][at])

    y = _plain_ffn(x[None], take("sg", None), take("su", None), take("sd", None), c["codes"])[0]
    e = idx.long().reshape(-1)
    o = _plain_ffn(x.repeat_interleave(k, 0)[:, None], take("wg", e), take("wu", e), take("wd", e), c["codes"])
    y = (y + (o.view(R, k, H) * w[:, :, None]).sum(1)).to(torch.bfloat16)
    return y if c["given"] else (y, idx, w)


def run(s):
    c = s["case"]
    if own:
        from sparse_moe_layer_row_gb300 import moe_block as mb
        if c["op"] == "norm":
            mb.moe_add_rmsnorm(s["x"], s["w"], EPS, residual=s.get("res"), total=s.get("sum"),
                               y=s.get("y"), codes=s.get("codes"), scales=s.get("scales"))
            return [s[n] for n in ("sum", "y", "codes", "scales") if n in s]
        if c["op"] == "quantize":
            mb.moe_i8_quantize(s["x"], s["codes"], s["scales"])
            return s["codes"], s["scales"]
        if c["op"] == "gemm":
            mb.moe_i8_gemm(s["xq"], s["xs"], s["wq"], s["ws"], s["y"], s["ws_mem"])
            return s["y"]
        if c["given"]:
            return s["layer"].token_forward(s["x"], s["idx"], s["w"], y=s["y"])
        s["layer"].token_pass(s["x"], topk_idx=s["idx"], topk_w=s["w"], y=s["y"])
        return s["y"], s["idx"], s["w"]
    if c["op"] == "norm":
        return _plain_norm(s)
    if c["op"] == "quantize":
        return _rows_i8(s["x"])
    if c["op"] == "gemm":
        acc = s["xq"].float() @ s["wq"].float().t()
        return (acc * (s["xs"][:, None] * s["ws"])).to(_DTYPES[c["out"]])
    return _plain_token(s)


# ------------------------------------------------------------------------------ work

def work(case):
    c = case
    R = c["R"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if c["op"] == "norm":
        H = c["H"]
        n = R * H * size[c["dtype"]] + H * size[c["weight"]]
        if c["residual"] != "none":
            n += 2 * R * H * size[c["residual"]]
        n += R * H * size[c["dtype"]] if c["out"] == "same" else R * H
        n += 4 * R * -(-H // BLOCK) if c["out"] == "e4m3" else 4 * R if c["out"] == "i8" else 0
        return {"bytes": n, "flops": 6 * R * H}
    if c["op"] == "quantize":
        K = c["K"]
        return {"bytes": R * K * (size[c["dtype"]] + 1) + 4 * R, "flops": 3 * R * K}
    if c["op"] == "gemm":
        N, K = c["N"], c["K"]
        return {"bytes": R * K + N * K + 4 * (R + N) + R * N * size[c["out"]], "flops": 2 * R * N * K}
    H, E, k, I, Is = (c[n] for n in ("H", "E", "k", "I", "Is"))
    touched = E * (1.0 - (1.0 - k / E) ** R)   # experts that the rows' routing touches, on average
    each = 2.0 if c["codes"] == "bf16" else 1.0 + 4.0 / (BLOCK * BLOCK)
    route = 0 if c["given"] else 2 * E * H
    return {"bytes": (touched * I + Is) * 3 * H * each + route + 4 * R * H + 8 * R * k,
            "flops": 6 * R * H * (k * I + Is) + (0 if c["given"] else 2 * R * E * H)}


# -------------------------------------------------------------------- 64-bit values

def _round_e4m3(v):
    """Nearest e4m3 value of |v| <= 448 (halves to the even code), in 64 bits."""
    t = [m / 8 * 2.0 ** -6 for m in range(8)]
    t += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    t = torch.tensor(t[:127], dtype=torch.float64, device=v.device)   # 0 .. 448
    a = v.abs().contiguous()
    hi = torch.searchsorted(t, a).clamp(1, 126)
    lo = hi - 1
    mid = (t[lo] + t[hi]) / 2
    r = torch.where((a > mid) | ((a == mid) & (hi % 2 == 0)), t[hi], t[lo])
    return torch.where(v < 0, -r, r)


def _exact_e4m3(v):
    """Rows in 64 bits -> codes, and the largest magnitude of each block [blocks, R]."""
    codes, largest = torch.empty_like(v), []
    for b in range(0, v.shape[1], BLOCK):
        u = v[:, b:b + BLOCK]
        a = u.abs().max(dim=1).values.clamp_min(AMAX_MIN)
        codes[:, b:b + BLOCK] = _round_e4m3(FP8_MAX * u / a[:, None])
        largest.append(a)
    return codes, torch.stack(largest)


def _exact_norm(c, s):
    r = s["x"].double()
    out = []
    if c["residual"] != "none":
        total = r + s["res"].double()
        out.append(total)
        r = total.to(s["res"].dtype).double()   # the norm is that of the sum as it is stored
    rstd = torch.rsqrt(torch.mean(r ** 2, dim=1) + EPS)
    v = r * s["w"].double() * rstd[:, None]
    if c["out"] == "same":
        return out + [v]
    if c["out"] == "e4m3":
        codes, a = _exact_e4m3(v)
        return out + [codes, a / FP8_MAX]
    a = v.abs().max(dim=1).values
    return out + [torch.round(I8_MAX * v / a[:, None]).to(torch.int8), a / I8_MAX]


def _exact_matrix(s, n, at=None):
    q, sc = s[n], s[n + "s"]
    if at is not None:
        q, sc = q[at], None if sc is None else sc[at]
    w = q.double()
    if sc is not None:
        for i in range(sc.shape[0]):
            for j in range(sc.shape[1]):
                w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= sc[i, j].double()
    return w


def _exact_rows(x):
    q, a = _exact_e4m3(x)
    for b in range(a.shape[0]):
        q[:, b * BLOCK:(b + 1) * BLOCK] *= (a[b] / FP8_MAX)[:, None]
    return q


def _exact_token(c, s):
    R, k = c["R"], c["k"]
    x, idx, w = s["x"].double(), s["idx"], s["w"]
    if not c["given"]:
        z = torch.einsum("rh,eh->re", x, s["router"].double())
        idx = z.argsort(dim=1, descending=True, stable=True)[:, :k].to(torch.int32)
        w = torch.softmax(z.gather(1, idx.long()), dim=1)
    rounded = _exact_rows if c["codes"] == "e4m3" else (lambda v: v)
    x = rounded(x)

    def ffn(v, names, at=None):
        wg, wu, wd = (_exact_matrix(s, n, at) for n in names)
        g = v @ wg.t()
        return rounded(g * torch.sigmoid(g) * (v @ wu.t())) @ wd.t()

    y = ffn(x, ("sg", "su", "sd"))
    for r in range(R):
        for j in range(k):
            y[r] += w[r, j].double() * ffn(x[r:r + 1], ("wg", "wu", "wd"), int(idx[r, j]))[0]
    return y if c["given"] else (y, idx, w)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    if c["op"] == "quantize":
        x = s["x"].double()
        a = x.abs().max(dim=1).values.clamp_min(AMAX_MIN)
        return torch.round(I8_MAX * x / a[:, None]).to(torch.int8), a / I8_MAX
    if c["op"] == "gemm":
        return (s["xs"].double()[:, None] * s["xq"].double()) @ (s["ws"].double()[:, None] * s["wq"].double()).t()
    return _exact_token(c, s)
