"""The 8-bit linear products and the token log-probabilities of the library, as cases to measure.

Four operators: the quantisation of rows to int8 (activations by token, weights by output channel), the
int8 matrix product with its fused epilogues, the log-probabilities of given tokens with entropy and top
alternatives, and the gradient of those log-probabilities and entropies. `run` computes them in elementary
torch operations where `own` is false and through the library's entry points where it is true.
"""
import math

import torch

own = False

DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16}
LARGEST = {"quantize": 50257 * 1024, "matmul": 16384 * 2304 * 768, "logprobs": 8192 * 50304, "grad": 4096 * 50304}


def listed():
    return [
        # one token's activations before a linear layer of the 124M model, batch of one
        {"name": "quantize-one-token", "op": "quantize", "rows": 1, "K": 768, "pad": 0, "dtype": "bf16"},
        # the MLP's inner activations of the XL model (4 x 1024 tokens)
        {"name": "quantize-xl-mlp", "op": "quantize", "rows": 4096, "K": 6400, "pad": 0, "dtype": "bf16"},
        # the tied embedding of the medium model, unpadded vocabulary, quantised once from the fp32 weights
        {"name": "quantize-medium-wte", "op": "quantize", "rows": 50257, "K": 1024, "pad": 0, "dtype": "fp32"},
        # lm_head of one token in a generation loop: weights streamed once
        {"name": "matmul-decode-lm-head", "op": "matmul", "M": 1, "N": 50304, "K": 768, "pad": 0, "epilogue": "store",
         "out": "bf16"},
        # attention projection plus residual of a ragged batch of prompts, XL width, an inner size that fills no tile
        {"name": "matmul-ragged-resid", "op": "matmul", "M": 333, "N": 1600, "K": 1599, "pad": 1,
         "epilogue": "bias_resid", "out": "fp32"},
        # c_attn of the 124M model over 16 x 1024 tokens
        {"name": "matmul-124m-qkv", "op": "matmul", "M": 16384, "N": 2304, "K": 768, "pad": 0, "epilogue": "bias",
         "out": "bf16"},
        # c_fc with its GELU of the XL model over 2 x 1024 tokens
        {"name": "matmul-xl-fc-gelu", "op": "matmul", "M": 2048, "N": 6400, "K": 1600, "pad": 0,
         "epilogue": "bias_gelu", "out": "bf16"},
        # the drawn token of a generation loop, with five alternatives, at the draw's temperature
        {"name": "logprobs-one-token", "op": "logprobs", "rows": 1, "V": 50257, "pad": 47, "dtype": "bf16", "tau": 0.8,
         "top": 5, "ignored": 0.0, "masked": 0.0},
        # scoring 8 x 1024 tokens of text against the padded vocabulary
        {"name": "logprobs-score", "op": "logprobs", "rows": 8192, "V": 50257, "pad": 47, "dtype": "bf16", "tau": 1.0,
         "top": 5, "ignored": 0.25, "masked": 0.0},
        # fp32 logits of a small model with part of the vocabulary forbidden, twenty alternatives
        {"name": "logprobs-masked-fp32", "op": "logprobs", "rows": 1023, "V": 1021, "pad": 3, "dtype": "fp32",
         "tau": 0.7, "top": 20, "ignored": 0.1, "masked": 0.4},
        # the same small model's gradient
        {"name": "grad-masked-fp32", "op": "grad", "rows": 1023, "V": 1021, "pad": 3, "dtype": "fp32", "tau": 0.7,
         "ignored": 0.1, "masked": 0.4},
        # fine-tuning on drawn tokens, 4 x 1024 positions, the prompts' positions ignored
        {"name": "grad-finetune", "op": "grad", "rows": 4096, "V": 50257, "pad": 47, "dtype": "bf16", "tau": 1.0,
         "ignored": 0.25, "masked": 0.0},
    ]


def _log(rng, low, high):
    """A whole number between low and high, spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "logprobs", "grad"])
    most = LARGEST[op]
    if op == "quantize":
        K = _log(rng, 1, 8192)
        return {"op": op, "rows": _log(rng, 1, min(65536, most // K)), "K": K, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": rng.choice(["fp32", "bf16"])}
    if op == "matmul":
        # most often whole 16-byte rows (what the library's models have), else any inner size, with rows that
        # are padded to 16 bytes (pad) or packed
        K = _log(rng, 32, 8192)
        kind = rng.choice(["whole", "whole", "padded", "packed"])
        K = (K + 15) // 16 * 16 if kind == "whole" else K
        N = _log(rng, 8, 50304)
        M = _log(rng, 1, max(1, min(16384, most // (N * K))))
        if kind == "packed":   # rows that start anywhere: smaller sizes
            N = min(N, 4096)
            M = min(M, 2048)
        epilogue = rng.choice(["store", "bias", "bias_gelu", "bias_resid"])
        return {"op": op, "M": M, "N": N, "K": K, "pad": -K % 16 if kind == "padded" else 0, "epilogue": epilogue,
                "out": "fp32" if epilogue == "bias_resid" else rng.choice(["fp32", "bf16", "bf16"])}
    V = _log(rng, 32, 131072)
    dtype = rng.choice(["fp32", "bf16"])
    case = {"op": op, "rows": _log(rng, 1, min(16384, most // (V + 64) // (2 if dtype == "fp32" else 1))), "V": V,
            "pad": rng.choice([0, -V % 64, 1]), "dtype": dtype, "tau": rng.choice([1.0, 1.0, 0.7, 1.5]),
            "ignored": rng.choice([0.0, 0.25, 0.6]), "masked": rng.choice([0.0, 0.0, 0.5])}
    if op == "logprobs":
        case["top"] = rng.choice([0, 1, 5, 20, 32])
    return case


def _rows(shape, pad, dtype, fill):
    """A matrix of the given shape whose rows lie pad elements further apart than they are long."""
    rows, cols = shape
    whole = torch.zeros((rows, cols + pad), dtype=dtype, device="cuda")
    part = whole[:, :cols]
    part.copy_(fill)
    return part


def _codes(x):
    """The definition of the quantisation, for weights that a program has laid out before the calls."""
    amax = x.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, torch.round(127.0 * x.double() / amax.double()), 0.0)
    return q, (amax / 127.0).reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    c = dict(case)
    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    op = c["op"]
    if op == "quantize":
        # activations have a few large channels; weights are near normal
        big = 1.0 + 9.0 * (uniform(c["K"]) > 0.99)
        s["x"] = _rows((c["rows"], c["K"]), c["pad"], DTYPE[c["dtype"]], normal(c["rows"], c["K"]) * big)
        s["q"] = torch.empty((c["rows"], c["K"]), dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(c["rows"], device="cuda")
    elif op == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        a, s["a_scale"] = _codes(normal(M, K))
        b, s["b_scale"] = _codes(normal(N, K) * 0.02)
        s["a"] = _rows((M, K), c["pad"], torch.int8, a)
        s["b"] = _rows((N, K), c["pad"], torch.int8, b)
        s["bias"] = normal(N) * 0.1 if c["epilogue"] != "store" else None
        s["resid"] = normal(M, N) if c["epilogue"] == "bias_resid" else None
        s["out"] = torch.empty((M, N), dtype=DTYPE[c["out"]], device="cuda")
    else:
        R, V = c["rows"], c["V"]
        # logits as a language model gives them: a wide bulk and one favoured token, which is the target of half
        # the rows; forbidden tokens are -inf, and every 16th such row has nothing left
        x = normal(R, V) * 2.5
        liked = (uniform(R) * V).long().clamp_(max=V - 1)
        x.scatter_add_(1, liked[:, None], 4.0 + 8.0 * uniform(R, 1))
        if c["masked"] > 0:
            x.masked_fill_(uniform(R, V) < c["masked"], -math.inf)
            x[5::16] = -math.inf
        x = _rows((R, V), c["pad"], DTYPE[c["dtype"]], x)
        any_token = (uniform(R) * V).long().clamp_(max=V - 1)
        targets = torch.where(uniform(R) < 0.5, liked, any_token)
        targets = torch.where(uniform(R) < c["ignored"], -1, targets).to(torch.int32)
        s["x"], s["targets"] = x, targets
        if op == "logprobs":
            for name in ("logp", "entropy", "lse"):
                s[name] = torch.empty(R, device="cuda")
            s["k"] = min(c["top"], V)
            s["top_ids"] = torch.empty((R, s["k"]), dtype=torch.int32, device="cuda") if s["k"] else None
            s["top_logp"] = torch.empty((R, s["k"]), device="cuda") if s["k"] else None
        else:
            z = x.double() / c["tau"] if R * V <= 1 << 26 else x.float() / c["tau"]
            lse = torch.logsumexp(z, 1)
            d = (z - lse[:, None]).nan_to_num_(nan=-math.inf)
            s["entropy"] = -(torch.exp(d) * d.clamp(min=-1e4)).sum(1).float()
            s["lse"] = lse.float()
            weight = (targets >= 0).float()
            s["dlogp"] = normal(R) / R
            s["dentropy"] = weight * 0.01 / R
            s["dx"] = torch.zeros((R, V + c["pad"]), dtype=x.dtype, device="cuda")[:, :V]
    return s


def run(state):
    c = state["case"]
    if own:
        return _library(state, c)
    return {"quantize": _quantize, "matmul": _matmul, "logprobs": _logprobs, "grad": _grad}[c["op"]](state, c)


def _library(s, c):
    from decoder_only_transformer_sm_b200 import native
    if c["op"] == "quantize":
        native.quantize_rows(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if c["op"] == "matmul":
        native.matmul_i8(s["a"], s["a_scale"], s["b"], s["b_scale"], s["out"], epilogue=c["epilogue"], bias=s["bias"],
                         resid=s["resid"], status=s["status"])
        return {"out": s["out"]}
    if c["op"] == "logprobs":
        native.token_logprobs(s["x"], c["V"], c["tau"], targets=s["targets"], logp=s["logp"], entropy=s["entropy"],
                              lse=s["lse"], top_ids=s["top_ids"], top_logp=s["top_logp"], status=s["status"])
        got = {name: s[name] for name in ("logp", "entropy", "lse")}
        return {**got, "top_ids": s["top_ids"], "top_logp": s["top_logp"]} if s["k"] else got
    native.token_logprobs_bwd(s["x"], c["V"], c["tau"], s["lse"], s["dx"], targets=s["targets"], dlogp=s["dlogp"],
                              entropy=s["entropy"], dentropy=s["dentropy"], status=s["status"])
    return {"dx": s["dx"]}


def _quantize(s, c):
    # the quotient in 64 bits: which code a value gets is decided at borders between two whole numbers
    x = s["x"].float()
    amax = x.abs().amax(1)
    fine = torch.isfinite(amax)
    scale = torch.where(fine, amax / 127.0, math.nan)
    live = (fine & (amax > 0))[:, None]
    q = torch.round(127.0 * x.double() / amax.double()[:, None])
    return {"q": torch.where(live, q, 0.0).to(torch.int8), "scale": scale}


def _matmul(s, c):
    u = (s["a"].float() @ s["b"].float().t()) * s["a_scale"][:, None] * s["b_scale"]
    if s["bias"] is not None:
        u = u + s["bias"]
    if c["epilogue"] == "bias_gelu":
        u = 0.5 * u * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (u + 0.044715 * u * u * u)))
    if s["resid"] is not None:
        u = s["resid"] + u
    return {"out": u.to(s["out"].dtype)}


def _logprobs(s, c):
    z = s["x"].float() / c["tau"]
    top = z.amax(1)
    empty, bad = top == -math.inf, ~(top < math.inf)
    d = z - torch.where(empty | bad, 0.0, top)[:, None]
    e = torch.exp(d)
    total = e.sum(1)
    log_total = torch.log(total)
    entropy = log_total - torch.where(e > 0, e * d, 0.0).sum(1) / total
    t = s["targets"].long()
    logp = torch.gather(d, 1, t.clamp(min=0)[:, None])[:, 0] - log_total

    def settle(v, nothing):
        return torch.where(bad, math.nan, torch.where(empty, nothing, v))

    got = {"logp": torch.where(t < 0, 0.0, settle(logp, -math.inf)), "entropy": settle(entropy, 0.0),
           "lse": settle(top + log_total, -math.inf)}
    if s["k"]:
        # one whole number orders values and, among equal ones, indices from the lowest
        bits = (s["x"].float() + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
        order = torch.where(torch.isnan(s["x"]), 0x7FFFFFFF, order)
        key = order * (1 << 24) + ((1 << 24) - 1 - torch.arange(c["V"], device="cuda"))
        best = torch.topk(key, s["k"], dim=1, sorted=True).indices
        got["top_ids"] = best.to(torch.int32)
        got["top_logp"] = settle((torch.gather(d, 1, best) - log_total[:, None]).t(), -math.inf).t().contiguous()
    return got


def _grad(s, c):
    d = s["x"].float() / c["tau"] - s["lse"][:, None]
    p = torch.where(s["lse"][:, None] == -math.inf, 0.0, torch.exp(d))
    t = s["targets"].long()
    g = torch.where(t < 0, 0.0, s["dlogp"])
    h = s["dentropy"]
    dz = torch.where(p == 0, 0.0, -p * (g[:, None] + h[:, None] * (d + s["entropy"][:, None])))
    dz.scatter_add_(1, t.clamp(min=0)[:, None], torch.where(s["lse"] == -math.inf, 0.0, g)[:, None])
    dz = torch.where(((g == 0) & (h == 0))[:, None], 0.0, dz)
    return {"dx": (dz / c["tau"]).to(s["x"].dtype)}


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * (5 if c["dtype"] == "fp32" else 3) + 4 * c["rows"], "flops": 3 * n}
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        es = 4 if c["out"] == "fp32" else 2
        more = (4 * N if c["epilogue"] != "store" else 0) + (4 * M * N if c["epilogue"] == "bias_resid" else 0)
        return {"bytes": (M + N) * (K + 4) + M * N * es + more, "flops": 2 * M * N * K}
    es = 4 if c["dtype"] == "fp32" else 2
    n = c["rows"] * c["V"]
    if c["op"] == "logprobs":
        return {"bytes": n * es + c["rows"] * (16 + 8 * c["top"]), "flops": 6 * n}
    return {"bytes": int(n * es * (2.0 - c["ignored"])) + 20 * c["rows"], "flops": 8 * n}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        x = s["x"].double()
        largest = torch.max(x.abs(), dim=1).values
        step = torch.where(largest > 0, largest, 1.0) / 127.0
        ratio = x / torch.where(largest > 0, largest, 1.0)[:, None] * 127.0
        # a value whose quotient the division rounds to a border is settled by whole multiples
        low = torch.floor(ratio)
        above = (254.0 * x - (2.0 * low + 1.0) * torch.where(largest > 0, largest, 1.0)[:, None])
        q = torch.where(above > 0, low + 1, torch.where(above < 0, low, low + torch.remainder(low, 2.0)))
        return {"q": q.to(torch.int8), "scale": torch.where(largest > 0, step, 0.0)}
    if c["op"] == "matmul":
        u = torch.matmul(s["a"].double(), s["b"].double().t())
        u.mul_(torch.outer(s["a_scale"].double(), s["b_scale"].double()))
        if c["epilogue"] != "store":
            u.add_(s["bias"].double())
        if c["epilogue"] == "bias_gelu":
            # 0.5 (1 + tanh y) is the logistic function of 2 y
            u = u * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (u + 0.044715 * u.pow(3)))
        if c["epilogue"] == "bias_resid":
            u.add_(s["resid"].double())
        return {"out": u}
    many = max(1, (1 << 26) // c["V"])
    parts = []
    for at in range(0, c["rows"], many):
        rows = slice(at, min(at + many, c["rows"]))
        z = s["x"][rows].double() / c["tau"]
        t = s["targets"][rows].long()
        if c["op"] == "logprobs":
            logp_all = torch.log_softmax(z, 1)
            nothing = torch.isneginf(z).all(1)
            logp_all[nothing] = -math.inf
            picked = logp_all.gather(1, t.clamp(min=0)[:, None])[:, 0]
            picked = torch.where(t < 0, 0.0, picked)
            terms = torch.special.entr(torch.exp(logp_all))
            part = {"logp": picked, "entropy": terms.sum(1), "lse": torch.logsumexp(z, 1)}
            if s["k"]:
                ids = torch.sort(s["x"][rows].float(), dim=1, descending=True, stable=True).indices[:, :s["k"]]
                part["top_ids"] = ids.to(torch.int32)
                part["top_logp"] = logp_all.gather(1, ids)
        else:
            lse, H = s["lse"][rows].double()[:, None], s["entropy"][rows].double()[:, None]
            g = torch.where(t < 0, 0.0, s["dlogp"][rows].double())[:, None]
            h = s["dentropy"][rows].double()[:, None]
            logp = torch.where(torch.isneginf(lse), -math.inf, z - lse)
            p = torch.exp(logp)
            dz = h * (torch.special.entr(p) - p * H) - g * p
            one = torch.zeros_like(dz).scatter_(1, t.clamp(min=0)[:, None], 1.0)
            part = {"dx": torch.where(torch.isneginf(lse), 0.0, (dz + g * one) / c["tau"])}
        parts.append(part)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
