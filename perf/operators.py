"""Measured cases of the layer operators around the verify step: attention over a
shared prefix and a paged cache, the residual RMSNorm with an 8-bit output, and the
matrix product with bias, activation and residual.

``run`` computes a case either in plain torch operations (``own`` false) or through the
library's calls (``own`` true); ``exact`` computes it from the definition in 64 bits.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest scale of an 8-bit row
EPS = 1e-5

NONE, RELU, SILU, GELU, GELU_TANH = range(5)  # activations
F32, BF16, E4M3 = range(3)  # types, as the library numbers them
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
CODES = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
SIZES = {"f32": 4, "bf16": 2, "e4m3": 1}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def _attn(B, K, kmin, prefix, own_min, own_max, hq, hkv, d, page, fused):
    return {"op": "attn", "B": B, "K": K, "kmin": kmin, "prefix": prefix, "own_min": own_min,
            "own_max": own_max, "hq": hq, "hkv": hkv, "d": d, "page": page, "fused": fused}


def _norm(M, H, dtype, out, res):
    return {"op": "norm", "M": M, "H": H, "dtype": dtype, "out": out, "res": res}


def _linear(M, N, K, dtype, out, act, bias, res):
    return {"op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "out": out, "act": act,
            "bias": bias, "res": res}


def listed():
    return [
        # one sequence, one new token: the latency of a decode step
        dict(_attn(1, 0, 0, 256, 100, 100, 32, 8, 128, 16, False), name="attn_token"),
        # 64 sequences of 7 drafts behind a common instruction, pages of 16 tokens
        dict(_attn(64, 7, 7, 2048, 100, 511, 32, 8, 128, 16, True), name="attn_round"),
        # the headline verify batch (256 sequences, 2 to 8 drafts, 128 to 4096 own tokens)
        # behind a long shared document
        dict(_attn(256, 8, 2, 16384, 128, 4096, 32, 8, 128, 16, True), name="attn_document"),
        # a small model with a key head for every query head, sequences that have just
        # begun (some with no token yet), a prefix that ends inside a page of 7 tokens
        dict(_attn(33, 5, 0, 1003, 0, 300, 12, 12, 64, 7, False), name="attn_odd"),
        # one token's hidden state before an 8-bit product
        dict(_norm(1, 4096, "bf16", "e4m3", True), name="norm_token"),
        # every position of the headline verify batch (256 x 9)
        dict(_norm(2304, 4096, "bf16", "e4m3", True), name="norm_round"),
        # a prompt's positions with the residual stream kept in 32 bits
        dict(_norm(16384, 8192, "f32", "bf16", True), name="norm_prompt"),
        # a draft head's residual block on one token
        dict(_linear(1, 4096, 4096, "bf16", "bf16", SILU, True, True), name="linear_token"),
        # sixteen sequences' single tokens, 8-bit weights
        dict(_linear(16, 8192, 8192, "e4m3", "bf16", NONE, True, False), name="linear_step"),
        # 64 x 8 positions of a verify round into a feed-forward block, 8-bit
        dict(_linear(512, 16384, 4096, "e4m3", "bf16", GELU, False, False), name="linear_round"),
        # a prompt's positions through an output projection onto the residual stream
        dict(_linear(8192, 4096, 4096, "bf16", "bf16", NONE, True, True), name="linear_prompt"),
        # a ragged batch and an odd width, 32-bit output
        dict(_linear(77, 1999, 1000, "bf16", "f32", GELU_TANH, True, True), name="linear_odd"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "norm", "linear"])
    if op == "attn":
        while True:
            hkv = rng.choice([1, 2, 4, 8, 12])
            hq = hkv * rng.choice([1, 2, 4, 5, 8])
            K = rng.randint(0, 12)
            own_max = _log(rng, 1, 4096)
            c = _attn(_log(rng, 1, 256), K, rng.randint(0, K), rng.choice([0, _log(rng, 1, 16384)]),
                      rng.randint(0, own_max), own_max, hq, hkv, rng.choice([64, 128]),
                      rng.choice([1, 7, 16, 32, 64]), rng.choice([False, True]))
            # no more queries times keys than the largest listed case
            keys = c["prefix"] + c["own_max"] + K
            if c["B"] * (K + 1) * hq * keys <= 256 * 6 * 32 * 18000 and hkv <= 8 * 256 // c["B"]:
                return c
    if op == "norm":
        H = _log(rng, 16, 16384)
        M = max(1, min(_log(rng, 1, 16384), 16384 * 8192 // H))
        return _norm(M, H, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "e4m3"]),
                     rng.choice([False, True]))
    while True:
        dtype = rng.choice(["bf16", "e4m3"])
        K = _log(rng, 16, 1024) * 16
        M, N = _log(rng, 1, 8192), _log(rng, 16, 32000)
        if M * N * K <= 8192 * 4096 * 4096 and N * K <= 1 << 28:
            return _linear(M, N, K, dtype, rng.choice(["bf16", "bf16", "f32"]), rng.randrange(5),
                           rng.choice([False, True]), rng.choice([False, True]))


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def integers(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)

    if case["op"] == "attn":
        return _prepare_attn(case, g, normal, integers)
    if case["op"] == "norm":
        t = TYPES[case["dtype"]]
        M, H = case["M"], case["H"]
        return {"case": case, "x": normal(M, H, dtype=t),
                "res": normal(M, H, scale=3.0, dtype=t) if case["res"] else None,
                "w": (1.0 + 0.02 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)}
    M, N, K = case["M"], case["N"], case["K"]
    s = {"case": case, "sx": None, "sw": None}
    x, W = normal(M, K, dtype=torch.float32), normal(N, K, scale=K ** -0.5, dtype=torch.float32)
    if case["dtype"] == "e4m3":  # an 8-bit row and its scale, as the norm leaves them
        s["sx"], s["sw"] = x.abs().amax(1) / E4M3_MAX, W.abs().amax(1) / E4M3_MAX
        x, W = x / s["sx"][:, None], W / s["sw"][:, None]
    t = TYPES[case["dtype"]]
    s["x"], s["W"] = x.to(t), W.to(t)
    s["bias"] = normal(N, scale=0.1) if case["bias"] else None
    s["res"] = normal(M, N, dtype=TYPES[case["out"]]) if case["res"] else None
    return s


def _prepare_attn(case, g, normal, integers):
    B, K, hq, hkv, d, page = (case[k] for k in ("B", "K", "hq", "hkv", "d", "page"))
    lens = integers(case["own_min"], case["own_max"], B)
    k = integers(case["kmin"], K, B)
    used = (lens + k + page - 1) // page
    max_pages = max(1, -(-(case["own_max"] + K) // page))
    pre = -(-case["prefix"] // page)
    pages = pre + B * max_pages
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = ids[pre:].reshape(B, max_pages)
    table = torch.where(torch.arange(max_pages, device="cuda")[None] < used[:, None], table, -1)
    # queries beside their keys and values where one product made all three
    wide = (hq + 2 * hkv) * d if case["fused"] else hq * d
    q = normal(B, K + 1, wide)
    return {"case": case, "q": q, "kp": normal(pages, page, hkv, d), "vp": normal(pages, page, hkv, d),
            "prefix_pages": ids[:pre].contiguous(), "table": table.contiguous(), "lens": lens, "k": k,
            "scale": d ** -0.5}


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _own_attn, "norm": _own_norm, "linear": _own_linear}[op](state)
    return {"attn": _plain_attn, "norm": _plain_norm, "linear": _plain_linear}[op](state)


def _own_attn(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    B, K, hq, hkv, d = (c[k] for k in ("B", "K", "hq", "hkv", "d"))
    max_pages = s["table"].shape[1]
    if "ws" not in s:  # a program keeps its workspace and its buffers
        s["ws"] = torch.zeros(sb.sv_prefix_attention_workspace_size(
            B, K, hq, hkv, d, c["prefix"], max_pages * c["page"]), dtype=torch.uint8, device="cuda")
        # rows behind a sequence's last draft stay as they are
        s["out"] = torch.zeros(B, K + 1, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(B, K + 1, hq, device="cuda")
    row = s["q"].shape[2]
    sb.sv_prefix_attention(s["q"], (K + 1) * row, row, d, s["kp"], s["vp"], 0, 0, 0, s["kp"].shape[0],
                           c["page"], s["prefix_pages"], c["prefix"], s["table"], max_pages, s["lens"],
                           s["k"], s["scale"], s["out"], 0, 0, 0, s["lse"], BF16, B, K, hq, hkv, d,
                           s["ws"], s["ws"].numel())
    return {"out": s["out"], "lse": s["lse"]}


def _own_norm(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    M, H = c["M"], c["H"]
    q8 = c["out"] == "e4m3"
    y = torch.empty(M, H, dtype=TYPES[c["out"]], device="cuda")
    scale = torch.empty(M, device="cuda") if q8 else None
    summed = torch.empty_like(s["x"]) if c["res"] else None
    sb.sv_rmsnorm_residual(s["x"], 0, s["res"], 0, s["w"], EPS, summed, 0, CODES[c["dtype"]], y, 0,
                           CODES[c["out"]], scale, M, H)
    return {"y": y, "scale": scale, "sum": summed}


def _own_linear(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    if "ws" not in s:
        s["ws"] = torch.zeros(sb.sv_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    ws = s["ws"]
    out = torch.empty(M, N, dtype=TYPES[c["out"]], device="cuda")
    sb.sv_linear(s["x"], 0, s["sx"], s["W"], 0, s["sw"], CODES[c["dtype"]], s["bias"], s["res"], 0, c["act"],
                 out, 0, CODES[c["out"]], M, N, K, ws, ws.numel())
    return out


def _plain_attn(s):
    c = s["case"]
    B, K, hq, hkv, d, page, P = (c[k] for k in ("B", "K", "hq", "hkv", "d", "page", "prefix"))
    G, Q = hq // hkv, K + 1
    q = s["q"][..., :hq * d].float().reshape(B, Q, hkv, G, d)
    q = q.permute(2, 0, 1, 3, 4) * s["scale"]                           # hkv B Q G d
    at = s["prefix_pages"].long()
    pk = s["kp"][at].float().reshape(-1, hkv, d)[:P].permute(1, 2, 0)   # hkv d P
    pv = s["vp"][at].float().reshape(-1, hkv, d)[:P].permute(1, 0, 2)   # hkv P d
    sp = (q.reshape(hkv, B * Q * G, d) @ pk).reshape(hkv, B, Q * G, P)
    own_pages = s["table"].long().clamp(min=0)                          # pages past a sequence's end are masked
    ok = s["kp"][own_pages].reshape(B, -1, hkv, d).permute(2, 0, 3, 1).float()
    ov = s["vp"][own_pages].reshape(B, -1, hkv, d).permute(2, 0, 1, 3).float()
    so = q.reshape(hkv, B, Q * G, d) @ ok                               # hkv B Q*G T
    i = torch.arange(Q, device="cuda")
    seen = torch.arange(so.shape[3], device="cuda")[None, None] < (s["lens"][:, None] + i)[..., None]
    so = so.masked_fill(~seen.repeat_interleave(G, 1), float("-inf"))
    m = so.amax(3, keepdim=True)
    m = torch.maximum(m, sp.amax(3, keepdim=True)) if P else m
    ref = torch.where(torch.isfinite(m), m, 0.0)
    wp, wo = (sp - ref).exp_(), (so - ref).exp_()
    total = wp.sum(3, keepdim=True) + wo.sum(3, keepdim=True)
    o = (wp.reshape(hkv, B * Q * G, P) @ pv).reshape(hkv, B, Q * G, d) + wo @ ov
    o = torch.where(total > 0, o / total, 0.0)
    lse = total.log() + ref
    valid = i[None] <= s["k"][:, None]                                  # rows past k_b are not computed
    o = o.reshape(hkv, B, Q, G, d).permute(1, 2, 0, 3, 4).reshape(B, Q, hq, d)
    lse = lse.reshape(hkv, B, Q, G).permute(1, 2, 0, 3).reshape(B, Q, hq)
    return {"out": torch.where(valid[..., None, None], o, 0.0).to(torch.bfloat16),
            "lse": torch.where(valid[..., None], lse, 0.0)}


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if s["res"] is not None:
        x = x + s["res"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["w"].float()
    summed = x.to(s["x"].dtype) if s["res"] is not None else None
    if c["out"] == "bf16":
        return {"y": y.to(torch.bfloat16), "scale": None, "sum": summed}
    scale = (y.abs().amax(1) / E4M3_MAX).clamp(min=TINY)
    return {"y": (y / scale[:, None]).to(torch.float8_e4m3fn), "scale": scale, "sum": summed}


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["W"].float().T
    if s["sx"] is not None:
        z = z * s["sx"][:, None] * s["sw"][None]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if c["act"] == RELU:
        z = z.clamp(min=0)
    elif c["act"] == SILU:
        z = z / (1 + torch.exp(-z))
    elif c["act"] == GELU:
        z = 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    elif c["act"] == GELU_TANH:
        z = 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if s["res"] is not None:
        z = z + s["res"].float()
    return z.to(TYPES[c["out"]])


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    if case["op"] == "attn":
        # lengths and draft counts at their mean over prepare()'s draws
        c = case
        rows = c["B"] * ((c["kmin"] + c["K"]) / 2 + 1)
        tail = (c["own_min"] + c["own_max"]) / 2
        k = (c["kmin"] + c["K"]) / 2
        own_keys = c["B"] * (tail + k)
        kv = (c["prefix"] + own_keys) * c["hkv"] * c["d"] * 2 * 2
        flops = 4 * c["hq"] * c["d"] * rows * (c["prefix"] + tail + k / 2)
        return {"bytes": kv + rows * c["hq"] * (c["d"] * 4 + 4), "flops": flops}
    if case["op"] == "norm":
        n, e = case["M"] * case["H"], SIZES[case["dtype"]]
        scales = case["M"] * 4 if case["out"] == "e4m3" else 0
        return {"bytes": n * (e * (3 if case["res"] else 1) + SIZES[case["out"]]) + case["H"] * 2 + scales,
                "flops": 6 * n}
    M, N, K, e = case["M"], case["N"], case["K"], SIZES[case["dtype"]]
    scales = (M + N) * 4 if case["dtype"] == "e4m3" else 0
    return {"bytes": (M + N) * K * e + scales + M * N * SIZES[case["out"]] * (2 if case["res"] else 1)
            + (N * 2 if case["bias"] else 0), "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](s)


def _exact_attn(s):
    """Sequence by sequence and position by position: a softmax over exactly the keys it sees."""
    c = s["case"]
    B, K, hq, hkv, d, P = (c[k] for k in ("B", "K", "hq", "hkv", "d", "prefix"))
    G = hq // hkv
    lens, k = s["lens"].tolist(), s["k"].tolist()
    out = torch.zeros(B, K + 1, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, K + 1, hq, dtype=torch.float64, device="cuda")

    def rows(pool, pages, n):
        return pool[pages.long()].reshape(-1, hkv, d)[:n].double()

    pk, pv = rows(s["kp"], s["prefix_pages"], P), rows(s["vp"], s["prefix_pages"], P)
    for b in range(B):
        used = -(-(lens[b] + k[b]) // c["page"])
        keys = torch.cat([pk, rows(s["kp"], s["table"][b, :used], lens[b] + k[b])])
        values = torch.cat([pv, rows(s["vp"], s["table"][b, :used], lens[b] + k[b])])
        q = s["q"][b, :, :hq * d].double().reshape(K + 1, hkv, G, d)
        for i in range(k[b] + 1):
            n = P + lens[b] + i
            if n == 0:
                lse[b, i] = -math.inf
                continue
            z = torch.einsum("hgd,nhd->hgn", q[i], keys[:n]) * s["scale"]
            lse[b, i] = torch.logsumexp(z, 2).reshape(hq)
            out[b, i] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, 2), values[:n]).reshape(hq, d)
    return {"out": out, "lse": lse}


def _exact_e4m3(v):
    """The nearest e4m3 values (3 bits behind the leading one, smallest step 2^-9), ties to even."""
    exponent = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(s):
    x = s["x"].double()
    total = x if s["res"] is None else x + s["res"].double()
    rms = (total * total).sum(1, keepdim=True).div(total.shape[1]).add(EPS).sqrt()
    y = total / rms * s["w"].double()
    summed = None if s["res"] is None else total
    if s["case"]["out"] == "bf16":
        return {"y": y, "scale": None, "sum": summed}
    scale = torch.clamp(y.abs().max(1).values / E4M3_MAX, min=TINY)
    return {"y": _exact_e4m3(y / scale[:, None]), "scale": scale, "sum": summed}


def _exact_linear(s):
    c = s["case"]
    x, W = s["x"].double(), s["W"].double()
    if s["sx"] is not None:
        x, W = x * s["sx"].double()[:, None], W * s["sw"].double()[:, None]
    z = torch.einsum("mk,nk->mn", x, W)
    if s["bias"] is not None:
        z += s["bias"].double()
    if c["act"] == RELU:
        z = torch.relu(z)
    elif c["act"] == SILU:
        z = z * torch.sigmoid(z)
    elif c["act"] == GELU:
        z = torch.nn.functional.gelu(z)
    elif c["act"] == GELU_TANH:
        z = torch.nn.functional.gelu(z, approximate="tanh")
    return z if s["res"] is None else z + s["res"].double()
