"""The 8-bit operators of the serving path: what is measured, and their plain forms.

  norm   nc_add_rmsnorm_fp8: residual add, RMSNorm, e4m3 output with a scale per 1 x 128 block
  quant  nc_quant_fp8: a matrix to e4m3 with a scale per 1 x 128 (activations) or 128 x 128 (weights) block
  gemm   nc_gemm_fp8: product of two such matrices with a fused epilogue
  mlp    norm, up-projection (relu^2 to 8 bits) and down-projection (residual add) in a row, as a block runs them

A block of values v with largest magnitude a is held as q = round_e4m3(448 v / a) and s = a / 448.
Activation scales are stored k-block-major, s[kb, m]; weight scales s[nb, kb].
"""
import math

import torch

own = False

EPILOGUES = ["store", "store_f32", "add", "relu2", "softcap", "relu2_fp8"]


def listed():
    return [
        # one decoded token of the depth-20 model (width 1280)
        {"name": "norm_token", "op": "norm", "M": 1, "C": 1280, "dtype": "bf16"},
        # an odd batch of prompt tokens, fp32 residual stream, the depth-32 width
        {"name": "norm_f32_ragged", "op": "norm", "M": 1023, "C": 2048, "dtype": "f32"},
        # prefill of 16 prompts of 2048 tokens at depth 20
        {"name": "norm_prefill", "op": "norm", "M": 32768, "C": 1280, "dtype": "bf16"},
        # attention output of an odd number of prompt tokens at the depth-24 width, before its projection
        {"name": "quant_rows", "op": "quant", "M": 5003, "C": 1536, "rows": 1, "dtype": "bf16"},
        # a depth-32 MLP weight from its fp32 master copy when the serving copy is made
        {"name": "quant_weight", "op": "quant", "M": 8192, "C": 2048, "rows": 128, "dtype": "f32"},
        # fused q, k, v projection of one decoded token at depth 20
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 1536, "K": 1280, "epi": "store"},
        # softcapped logits of 16 decoded rows over the 65,536-id vocabulary
        {"name": "gemm_head", "op": "gemm", "M": 16, "N": 65536, "K": 1280, "epi": "softcap"},
        # an odd number of tokens through the depth-24 down-projection onto the residual stream
        {"name": "gemm_add_ragged", "op": "gemm", "M": 333, "N": 1536, "K": 6144, "epi": "add"},
        # sizes that no tile divides, fp32 result
        {"name": "gemm_f32_odd", "op": "gemm", "M": 1001, "N": 1003, "K": 1040, "epi": "store_f32"},
        # up-projection of a prefill of 16 x 2048 tokens at depth 20, its relu^2 held in 8 bits
        {"name": "gemm_up", "op": "gemm", "M": 32768, "N": 5120, "K": 1280, "epi": "relu2_fp8"},
        # down-projection of 8 x 2048 tokens at depth 32 onto the residual stream
        {"name": "gemm_down", "op": "gemm", "M": 16384, "N": 2048, "K": 8192, "epi": "add"},
        # the whole MLP of one full-context prompt at depth 20
        {"name": "mlp_prompt", "op": "mlp", "M": 2048, "C": 1280, "F": 5120},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "gemm", "mlp"])
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 32768), "C": 16 * _log(rng, 4, 80),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "quant":
        return {"op": op, "M": _log(rng, 1, 16384), "C": 16 * _log(rng, 4, 128), "rows": rng.choice([1, 128]),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "mlp":
        C = 128 * rng.randint(2, 10)
        return {"op": op, "M": _log(rng, 1, 16384), "C": C, "F": 4 * C}
    while True:
        c = {"op": op, "M": _log(rng, 1, 32768), "N": _log(rng, 64, 8192), "K": 16 * _log(rng, 8, 512),
             "epi": rng.choice(EPILOGUES)}
        if c["M"] * c["N"] * c["K"] <= 2 ** 37:
            return c


# ---- shapes and work ----

def _up(n, m):
    return -(-n // m) * m


def _blocks(n):
    return -(-n // 128)


def work(case):
    if case["op"] == "norm":
        M, C, es = case["M"], case["C"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * (C * (3 * es + 1) + 4 * _blocks(C) + 4), "flops": 5 * M * C}
    if case["op"] == "quant":
        M, C, es = case["M"], case["C"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": M * C * (es + 1) + 4 * -(-M // case["rows"]) * _blocks(C), "flops": 3 * M * C}
    if case["op"] == "mlp":
        M, C, F = case["M"], case["C"], case["F"]
        return {"bytes": 6 * M * C + 2 * C * F + 8 * _blocks(C) * _blocks(F), "flops": 4 * M * C * F}
    M, N, K = case["M"], case["N"], case["K"]
    out = {"store": 2, "store_f32": 4, "add": 4, "relu2": 2, "softcap": 2, "relu2_fp8": 1 + 4 / 128}[case["epi"]]
    return {"bytes": M * K + N * K + 4 * _blocks(K) * (M + _blocks(N)) + out * M * N, "flops": 2 * M * N * K}


# ---- inputs ----

def _quantise(v, rows):
    """(q, s) of a float32 matrix by blocks of rows x 128: the form the operands are kept in."""
    R, K = v.shape
    Rb, Kb = -(-R // rows), _blocks(K)
    pad = torch.zeros(Rb * rows, Kb * 128, device=v.device)
    pad[:R, :K] = v
    b = pad.view(Rb, rows, Kb, 128)
    a = b.abs().amax(dim=(1, 3), keepdim=True)
    q = torch.where(a > 0, b * 448 / a, torch.zeros_like(b)).view(Rb * rows, Kb * 128)[:R, :K]
    s = (a / 448).view(Rb, Kb)
    return q.contiguous().to(torch.float8_e4m3fn), (s.t().contiguous() if rows == 1 else s)


def _rows(g, M, C):
    """Activations as a residual stream has them: a few channels far larger than the rest, rows of differing size."""
    x = torch.randn(M, C, device="cuda", generator=g)
    x *= torch.exp(torch.randn(1, C, device="cuda", generator=g))
    return x * torch.exp(0.5 * torch.randn(M, 1, device="cuda", generator=g))


def _weight(g, N, K):
    return torch.randn(N, K, device="cuda", generator=g) / math.sqrt(K)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _make(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "norm":
        x = _rows(g, case["M"], case["C"]).to(_type(case))
        return {"x": x, "res": (0.3 * torch.randn(x.shape, device="cuda", generator=g)).to(_type(case))}
    if op == "quant":
        v = _rows(g, case["M"], case["C"]) if case["rows"] == 1 else _weight(g, case["M"], case["C"])
        return {"x": v.to(_type(case))}
    if op == "mlp":
        M, C, F = case["M"], case["C"], case["F"]
        x = _rows(g, M, C).bfloat16()
        w1, s1 = _quantise(_weight(g, F, C), 128)
        w2, s2 = _quantise(_weight(g, C, F), 128)
        return {"x": x, "res": (0.3 * torch.randn(M, C, device="cuda", generator=g)).bfloat16(),
                "w1": w1, "s1": s1, "w2": w2, "s2": s2}
    M, N, K = case["M"], case["N"], case["K"]
    a, sa = _quantise(_rows(g, M, K), 1)
    b, sb = _quantise(_weight(g, N, K), 128)
    t = {"a": a, "sa": sa, "b": b, "sb": sb}
    if case["epi"] == "add":
        t["d"] = torch.randn(M, _up(N, 8), device="cuda", generator=g).bfloat16()
    return t


def prepare(case, seed):
    """Inputs, and the buffers that a program keeps for the results (rows padded to 16 bytes)."""
    s = {"case": case, **_make(case, seed)}
    op = case["op"]
    if op in ("norm", "quant"):
        M, C = case["M"], case["C"]
        s["q"] = torch.empty(M, C, dtype=torch.float8_e4m3fn, device="cuda")
        shape = (_blocks(C), M) if op == "norm" or case["rows"] == 1 else (-(-M // 128), _blocks(C))
        s["s"] = torch.empty(shape, dtype=torch.float32, device="cuda")
        if op == "norm":
            s["x_out"] = torch.empty_like(s["x"])
            s["r"] = torch.empty(M, dtype=torch.float32, device="cuda")
    elif op == "mlp":
        M, C, F = case["M"], case["C"], case["F"]
        s["x_out"] = torch.empty_like(s["x"])
        s["r"] = torch.empty(M, dtype=torch.float32, device="cuda")
        s["q"] = torch.empty(M, C, dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.empty(_blocks(C), M, dtype=torch.float32, device="cuda")
        s["h"] = torch.empty(M, F, dtype=torch.float8_e4m3fn, device="cuda")
        s["sh"] = torch.empty(_blocks(F), M, dtype=torch.float32, device="cuda")
    else:
        M, N = case["M"], case["N"]
        if case["epi"] == "relu2_fp8":
            s["d"] = torch.empty(M, _up(N, 16), dtype=torch.float8_e4m3fn, device="cuda")
            s["sd"] = torch.empty(_blocks(N), M, dtype=torch.float32, device="cuda")
        elif case["epi"] == "store_f32":
            s["d"] = torch.empty(M, _up(N, 4), dtype=torch.float32, device="cuda")
        elif case["epi"] != "add":
            s["d"] = torch.empty(M, _up(N, 8), dtype=torch.bfloat16, device="cuda")
    return s


# ---- the operators in their plain form ----

def _in_blocks(v):
    """[R, K] as [R, kb, 128], zeros behind K."""
    R, K = v.shape
    return torch.nn.functional.pad(v, (0, _blocks(K) * 128 - K)).view(R, _blocks(K), 128)


def _to_fp8(v):
    """1 x 128 blocks of fp32 rows: (448 v / a, a) with a per block."""
    b = _in_blocks(v)
    a = b.abs().amax(2, keepdim=True)
    q = torch.where(a > 0, b * 448 / a, torch.zeros_like(b))
    return q.view(v.shape[0], -1)[:, :v.shape[1]].to(torch.float8_e4m3fn), a[:, :, 0]


def _plain_norm(x, res):
    x = (x.float() + res.float()).to(x.dtype)
    v = x.float()
    r = torch.rsqrt(v.square().mean(1) + 2.0 ** -23)
    q, a = _to_fp8(v)
    return x, q, (a * r[:, None] / 448).t().contiguous(), r


def _values(q, s, rows):
    """fp32 values of a quantised matrix; s [kb, rows] (rows == 1) or [nb, kb]."""
    K = q.shape[1]
    if rows == 1:
        return q.float() * s.t().repeat_interleave(128, 1)[:, :K]
    return q.float() * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :K]


def _plain_product(a, sa, b, sb):
    return _values(a, sa, 1) @ _values(b, sb, 128).t()


def _plain_relu2_fp8(acc):
    q, a = _to_fp8(torch.relu(acc).square())
    return q, (a / 448).t().contiguous()


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return list(_plain_norm(s["x"], s["res"]))
    if op == "quant":
        v = s["x"].float()
        if case["rows"] == 1:
            q, a = _to_fp8(v)
            return [q, (a / 448).t().contiguous()]
        R = v.shape[0]
        b = _in_blocks(torch.nn.functional.pad(v, (0, 0, 0, _up(R, 128) - R)))
        b = b.view(-1, 128, b.shape[1], 128)
        a = b.abs().amax((1, 3), keepdim=True)
        q = torch.where(a > 0, b * 448 / a, torch.zeros_like(b)).view(_up(R, 128), -1)[:R, :v.shape[1]]
        return [q.to(torch.float8_e4m3fn), (a / 448)[:, 0, :, 0]]
    if op == "mlp":
        x, q, sq, _ = _plain_norm(s["x"], s["res"])
        h, sh = _plain_relu2_fp8(_plain_product(q, sq, s["w1"], s["s1"]))
        return (x.float() + _plain_product(h, sh, s["w2"], s["s2"])).bfloat16()
    acc = _plain_product(s["a"], s["sa"], s["b"], s["sb"])
    epi = case["epi"]
    if epi == "relu2_fp8":
        return list(_plain_relu2_fp8(acc))
    if epi == "store_f32":
        return acc
    if epi == "add":  # onto the residual stream, in place
        d = s["d"][:, :case["N"]]
        d.copy_(d.float() + acc)
        return d
    if epi == "relu2":
        acc = torch.relu(acc).square()
    elif epi == "softcap":
        acc = 15 * torch.tanh(acc / 15)
    return acc.bfloat16()


# ---- the framework's calls ----

def _own(s):
    import decoder_only_transformer_nanochat_b200 as nc
    st = torch.cuda.current_stream().cuda_stream

    def ok(rc):
        if rc != nc.NC_OK:
            raise nc.NcError(rc)

    def p(name):
        return s[name].data_ptr()

    case = s["case"]
    op = case["op"]
    if op == "norm":
        M, C = case["M"], case["C"]
        ok(nc.nc_add_rmsnorm_fp8(p("x"), p("res"), p("x_out"), p("q"), p("s"), M, p("r"), M, C,
                                 nc.NC_BF16 if case["dtype"] == "bf16" else nc.NC_F32, st))
        return [s["x_out"], s["q"], s["s"], s["r"]]
    if op == "quant":
        M, C = case["M"], case["C"]
        ok(nc.nc_quant_fp8(p("x"), C, p("q"), C, p("s"), s["s"].shape[1], M, C, case["rows"],
                           nc.NC_BF16 if case["dtype"] == "bf16" else nc.NC_F32, st))
        return [s["q"], s["s"]]
    if op == "mlp":
        M, C, F = case["M"], case["C"], case["F"]
        ok(nc.nc_add_rmsnorm_fp8(p("x"), p("res"), p("x_out"), p("q"), p("s"), M, p("r"), M, C, nc.NC_BF16, st))
        ok(nc.nc_gemm_fp8(p("q"), C, p("s"), M, p("w1"), C, p("s1"), _blocks(C), p("h"), F, p("sh"), M, M, F, C,
                          nc.NC_EPI_RELU2_FP8, st))
        ok(nc.nc_gemm_fp8(p("h"), F, p("sh"), M, p("w2"), F, p("s2"), _blocks(F), p("x_out"), C, None, 0, M, C, F,
                          nc.NC_EPI_ADD, st))
        return s["x_out"]
    M, N, K = case["M"], case["N"], case["K"]
    epi = case["epi"]
    q8 = epi == "relu2_fp8"
    ok(nc.nc_gemm_fp8(p("a"), K, p("sa"), M, p("b"), K, p("sb"), _blocks(K), p("d"), s["d"].shape[1],
                      p("sd") if q8 else None, M if q8 else 0, M, N, K, getattr(nc, "NC_EPI_" + epi.upper()), st))
    d = s["d"][:, :N]
    return [d, s["sd"]] if q8 else d


def run(state):
    return _own(state) if own else _plain(state)


# ---- 64 bits, from the definition ----

def _exact_blocks(v):
    """(448 v / a unrounded, a) by 1 x 128 blocks, one block at a time."""
    q, amax = torch.zeros_like(v), []
    for k in range(0, v.shape[1], 128):
        a = v[:, k:k + 128].abs().max(1).values
        q[:, k:k + 128] = 448 * v[:, k:k + 128] / a.clamp_min(1e-300)[:, None]
        amax.append(a)
    return q, torch.stack(amax)


def _exact_product(a, sa, b, sb):
    """sum over the blocks of their scales' product times their codes' product."""
    acc = torch.zeros(a.shape[0], b.shape[0], dtype=torch.float64, device=a.device)
    for i, k in enumerate(range(0, a.shape[1], 128)):
        part = a[:, k:k + 128].double() @ b[:, k:k + 128].double().t()
        rows = sb[:, i].double()[torch.arange(b.shape[0], device=a.device) // 128]
        acc += part * sa[i].double()[:, None] * rows
    return acc


def exact(case, seed):
    """What run() returns, in 64 bits; 8-bit codes as the value 448 v / a that they round."""
    t = _make(case, seed)
    op = case["op"]
    if op in ("norm", "mlp"):
        x = t["x"].double() + t["res"].double()
        kept = x.to(t["x"].dtype).double()  # the stream is held in its type: the norm reads that
        r = 1 / (kept.square().sum(1) / kept.shape[1] + 2.0 ** -23).sqrt()
        q, a = _exact_blocks(kept)
        if op == "norm":
            return [x, q, a * r / 448, r]
        h = _exact_product(q.float().to(torch.float8_e4m3fn), a * r / 448, t["w1"], t["s1"]).clamp_min(0) ** 2
        q, a = _exact_blocks(h)
        return kept + _exact_product(q.float().to(torch.float8_e4m3fn), a / 448, t["w2"], t["s2"])
    if op == "quant":
        v = t["x"].double()
        if case["rows"] == 1:
            q, a = _exact_blocks(v)
            return [q, a / 448]
        q, s = torch.zeros_like(v), []
        for n in range(0, v.shape[0], 128):
            strip = [v[n:n + 128, k:k + 128] for k in range(0, v.shape[1], 128)]
            amax = [b.abs().max() for b in strip]
            q[n:n + 128] = torch.cat([448 * b / a for b, a in zip(strip, amax)], 1)
            s.append(torch.stack(amax) / 448)
        return [q, torch.stack(s)]
    acc = _exact_product(t["a"], t["sa"], t["b"], t["sb"])
    epi = case["epi"]
    if epi == "relu2_fp8":
        q, a = _exact_blocks(acc.clamp_min(0) ** 2)
        return [q, a / 448]
    if epi == "add":
        return t["d"][:, :case["N"]].double() + acc
    if epi == "relu2":
        return acc.clamp_min(0) ** 2
    if epi == "softcap":
        return 15 * torch.tanh(acc / 15)
    return acc
