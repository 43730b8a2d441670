"""Measured cases of a draft held in 4 bits: attention over a 4-bit paged cache, the writing
and reading of that cache, matrix products with 4-bit weights, and the moves of cache pages
(free, fork, compact).

``run`` computes a case either in plain torch operations (``own`` false) or through the
library's calls (``own`` true); ``exact`` computes it from the definition in 64 bits.

A 4-bit row of D values is its codes c (0 to 15, the even value in a byte's low half), a bf16
scale s and a bf16 minimum m: value = m + s c.  A page holds for each key head the codes of K
and of V, token by token, then the (s, m) of K's tokens and of V's, padded to 16 bytes.
"""

import math

import torch

own = False

NONE, RELU, SILU, GELU, GELU_TANH = range(5)  # activations
F32, BF16 = 0, 1  # types, as the library numbers them
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CODES = {"f32": F32, "bf16": BF16}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def _attn(B, K, kmin, own_min, own_max, hq, hkv, d, page, window, sinks):
    return {"op": "attn", "B": B, "K": K, "kmin": kmin, "own_min": own_min, "own_max": own_max, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "window": window, "sinks": sinks}


def _append(B, T, nmin, start_max, hkv, d, page):
    return {"op": "append", "B": B, "T": T, "nmin": nmin, "start_max": start_max, "hkv": hkv, "d": d, "page": page}


def _linear(M, N, K, group, zeros, act, bias, res, out):
    return {"op": "linear", "M": M, "N": N, "K": K, "group": group, "zeros": zeros, "act": act, "bias": bias,
            "res": res, "out": out}


def _fork(B, F, sources, own_min, own_max, pools, page_bytes, page):
    return {"op": "fork", "B": B, "F": F, "sources": sources, "own_min": own_min, "own_max": own_max,
            "pools": pools, "page_bytes": page_bytes, "page": page}


def _compact(B, pages, live, pools, page_bytes, prefix):
    return {"op": "compact", "B": B, "pages": pages, "live": live, "pools": pools, "page_bytes": page_bytes,
            "prefix": prefix}


def listed():
    return [
        # one sequence, one new draft token: the latency of a draft step
        dict(_attn(1, 0, 0, 356, 356, 32, 8, 128, 16, 0, 0), name="kv4_token"),
        # a draft step of the headline verify batch (256 sequences of 128 to 4096 tokens)
        dict(_attn(256, 0, 0, 128, 4096, 32, 8, 128, 16, 0, 0), name="kv4_step"),
        # 64 long sequences that see the last 1024 tokens and the first 4, one to four positions
        dict(_attn(64, 3, 0, 512, 16384, 32, 8, 128, 16, 1024, 4), name="kv4_window"),
        # a small model with a key head for every query head, sequences that have just begun
        # (some with no token yet), pages of 7 tokens
        dict(_attn(33, 5, 0, 0, 300, 12, 12, 64, 7, 0, 0), name="kv4_odd"),
        # a round's tokens (the emitted one and its drafts) into the headline batch's cache
        dict(_append(256, 9, 1, 4096, 8, 128, 16), name="append_round"),
        # eight prompts, the cache behind a few tokens each
        dict(_append(8, 4096, 1024, 100, 8, 128, 16), name="append_prompt"),
        # one token into a feed-forward block
        dict(_linear(1, 16384, 4096, 128, False, SILU, False, False, "bf16"), name="w4_token"),
        # sixteen sequences' single tokens through a projection onto the residual stream
        dict(_linear(16, 8192, 8192, 64, True, NONE, True, True, "bf16"), name="w4_step"),
        # 64 sequences' single tokens into a feed-forward block
        dict(_linear(64, 16384, 4096, 128, True, GELU, False, False, "bf16"), name="w4_batch"),
        # a few rows, an odd width, small groups, 32-bit output
        dict(_linear(5, 1999, 1024, 32, True, GELU_TANH, True, True, "f32"), name="w4_odd"),
        # 64 continuations end and 64 others are forked into their rows, keys and values of 32 layers
        dict(_fork(256, 64, 16, 100, 255, 64, 16 * 8 * 128 * 2, 16), name="pages_fork"),
        # a half-empty pool of two 16-token page arrays is compacted
        dict(_compact(64, 4096, 2048, 2, 16 * 8 * 128 * 2, 8), name="pages_compact"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "linear", "linear", "fork", "compact"])
    if op == "attn":
        while True:
            hkv = rng.choice([1, 2, 4, 8, 12])
            hq = hkv * rng.choice([1, 2, 4, 5, 8])
            K = rng.choice([0, 0, rng.randint(1, 8)])
            own_max = _log(rng, 1, 32768)
            window = rng.choice([0, _log(rng, 1, 4096)])
            c = _attn(_log(rng, 1, 256), K, rng.randint(0, K), rng.randint(0, own_max), own_max, hq, hkv,
                      rng.choice([64, 128]), rng.choice([1, 7, 16, 16, 32, 64]), window,
                      rng.choice([0, 4, rng.randint(1, 64)]) if window else 0)
            # no more cache and no more scores than the largest listed case
            if (c["B"] * (own_max + K) * hkv <= 256 * 4096 * 8 and
                    c["B"] * (own_max + K) * hq * (K + 1) <= 256 * 4096 * 32):
                return c
    if op == "append":
        while True:
            hkv, T = rng.choice([1, 2, 4, 8, 12]), _log(rng, 1, 4096)
            c = _append(_log(rng, 1, 256), T, rng.randint(0, T), _log(rng, 1, 4096), hkv, rng.choice([64, 128]),
                        rng.choice([1, 7, 16, 16, 32, 64]))
            if c["B"] * T * hkv <= 8 * 4096 * 8 and c["B"] * (T + c["start_max"]) * hkv <= 256 * 4096 * 8:
                return c
    if op == "linear":
        while True:
            group = rng.choice([32, 64, 128])
            K = group * max(1, _log(rng, 128, 16384) // group)
            N, M = _log(rng, 16, 32000), _log(rng, 1, 64)
            if M * N * K <= 64 * 16384 * 4096 and N * K <= 1 << 27:
                return _linear(M, N, K, group, rng.choice([False, True]), rng.randrange(5),
                               rng.choice([False, True]), rng.choice([False, True]), rng.choice(["bf16", "bf16", "f32"]))
    if op == "fork":
        while True:
            own_max, page = _log(rng, 1, 1024), rng.choice([1, 7, 16, 32])
            F = _log(rng, 1, 64)
            B = 2 * F + _log(rng, 1, 128)
            c = _fork(B, F, rng.randint(1, F), rng.randint(0, own_max), own_max, _log(rng, 1, 64),
                      page * rng.choice([1, 2, 8]) * rng.choice([64, 128]) * 2, page)
            if c["pools"] * c["page_bytes"] * B * (own_max // page + 1) <= 1 << 31:
                return c
    while True:
        pages = _log(rng, 2, 8192)
        c = _compact(_log(rng, 1, 256), pages, rng.randint(1, pages), _log(rng, 1, 8),
                     rng.choice([1, 7, 16, 32]) * rng.choice([1, 2, 8]) * rng.choice([64, 128]) * 2, rng.choice([0, 8]))
        if pages * c["pools"] * c["page_bytes"] <= 4096 * 2 * 32768:
            return c


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _head_bytes(d, page):
    return -(-page * (d + 8) // 16) * 16


def _quantise(x):
    """Codes, scales and minima of rows of bf16 values (the last axis); in 64 bits, since quotients lie next to a
    border of their rounding."""
    x = x.double()
    low = x.amin(-1, keepdim=True)
    # (a quotient by a plain number becomes a product with its reciprocal, which misses ties)
    scale = ((x.amax(-1, keepdim=True) - low) / torch.full_like(low, 15)).to(torch.bfloat16)
    step = torch.where(scale > 0, scale.double(), 1.0)
    codes = torch.where(scale > 0, ((x - low) / step).round().clamp(0, 15), 0.0).to(torch.uint8)
    return codes, scale[..., 0], low[..., 0].to(torch.bfloat16)


def _pack(kv, hkv, d, page):
    """Pages [n][page_bytes] of keys and values [2][n][hkv][page][d]."""
    codes, scale, low = _quantise(kv)
    n = kv.shape[1]
    nibbles = (codes[..., 0::2] | (codes[..., 1::2] << 4)).permute(1, 2, 0, 3, 4).reshape(n, hkv, page * d)
    words = torch.stack([scale, low], -1).permute(1, 2, 0, 3, 4).reshape(n, hkv, page * 4).contiguous()
    body = torch.cat([nibbles, words.view(torch.uint8).reshape(n, hkv, page * 8)], -1)
    pad = _head_bytes(d, page) - body.shape[-1]
    return torch.nn.functional.pad(body, (0, pad)).reshape(n, -1)


def _unpack(pages, hkv, d, page, dtype):
    """Keys and values [2][n][hkv][page][d] of pages [n][page_bytes]."""
    n = pages.shape[0]
    body = pages.reshape(n, hkv, -1)
    codes = body[..., :page * d].reshape(n, hkv, 2, page, d // 2)
    words = body[..., page * d:page * (d + 8)].contiguous().view(torch.bfloat16).reshape(n, hkv, 2, page, 2)
    codes = torch.stack([codes & 15, codes >> 4], -1).reshape(n, hkv, 2, page, d)
    values = words[..., 1:].to(dtype) + words[..., :1].to(dtype) * codes.to(dtype)
    return values.permute(2, 0, 1, 3, 4)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 23)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def integers(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)

    def shuffled(n):
        return torch.randperm(n, generator=g, device="cuda").to(torch.int32)

    return {"attn": _prepare_attn, "append": _prepare_append, "linear": _prepare_linear, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, normal, integers, shuffled)


def _tables(used, max_pages, ids):
    """Block tables whose first `used` entries of each row are pages, and the rest -1."""
    table = ids.reshape(used.shape[0], max_pages)
    return torch.where(torch.arange(max_pages, device="cuda")[None] < used[:, None], table, -1).contiguous()


def _prepare_attn(case, normal, integers, shuffled):
    B, K, hq, hkv, d, page = (case[k] for k in ("B", "K", "hq", "hkv", "d", "page"))
    lens, k = integers(case["own_min"], case["own_max"], B), integers(case["kmin"], K, B)
    max_pages = max(1, -(-(case["own_max"] + K) // page))
    ids = shuffled(B * max_pages)
    # keys whose channels have offsets of their own, as rotary keys do
    kv = normal(2, B * max_pages, hkv, page, d) + normal(2, 1, hkv, 1, d, scale=0.5)
    return {"case": case, "q": normal(B, K + 1, hq, d), "pool": _pack(kv, hkv, d, page),
            "table": _tables((lens + k + page - 1) // page, max_pages, ids), "lens": lens, "k": k, "scale": d ** -0.5}


def _prepare_append(case, normal, integers, shuffled):
    B, T, hkv, d, page = (case[k] for k in ("B", "T", "hkv", "d", "page"))
    starts, n = integers(0, case["start_max"], B), integers(case["nmin"], T, B)
    max_pages = -(-(case["start_max"] + T) // page)
    pool = torch.zeros(B * max_pages, hkv * _head_bytes(d, page), dtype=torch.uint8, device="cuda")
    # keys and values beside each other, as one product made them
    return {"case": case, "kv": normal(B, T, 2, hkv, d), "pool": pool, "starts": starts, "n": n,
            "table": _tables((starts + n + page - 1) // page, max_pages, shuffled(B * max_pages)),
            "out": torch.zeros(2, B, T, hkv, d, dtype=torch.bfloat16, device="cuda")}


def _prepare_linear(case, normal, integers, shuffled):
    M, N, K, group = (case[k] for k in ("M", "N", "K", "group"))
    W = normal(N, K // group, group, scale=K ** -0.5, dtype=torch.float32)
    if case["zeros"]:
        low, high = W.amin(2).clamp(max=0), W.amax(2).clamp(min=0)
        scales = ((high - low) / 15).to(torch.bfloat16)
        zeros = (-low / scales.float()).round().clamp(0, 15)
    else:
        scales = (W.abs().amax(2) / 7).to(torch.bfloat16)
        zeros = torch.full_like(scales, 8.0, dtype=torch.float32)
    codes = (W / scales.float()[..., None] + zeros[..., None]).round().clamp(0, 15).to(torch.uint8).reshape(N, K)
    return {"case": case, "x": normal(M, K), "W": codes[:, 0::2] | (codes[:, 1::2] << 4), "scales": scales,
            "zeros": zeros.to(torch.uint8) if case["zeros"] else None,
            "bias": normal(N, scale=0.1) if case["bias"] else None,
            "res": normal(M, N, dtype=TYPES[case["out"]]) if case["res"] else None}


def _index(parts):
    """One int32 array of all index arrays, so that a pass can begin from the same ones, and its pieces' sizes."""
    return torch.cat([p.reshape(-1).to(torch.int32) for p in parts]), [tuple(p.shape) for p in parts]


def _views(flat, shapes):
    pieces = torch.split(flat, [math.prod(s) for s in shapes])
    return [p.view(s) for p, s in zip(pieces, shapes)]


def _pool_words(case, pages):
    # any values: pages are moved, not read
    words = torch.arange(case["pools"] * pages * case["page_bytes"] // 8, device="cuda")
    return (words * -7046029254386353131).view(case["pools"], pages, -1)


def _prepare_fork(case, normal, integers, shuffled):
    B, F, page = case["B"], case["F"], case["page"]
    lens = integers(case["own_min"], case["own_max"], B)
    max_pages = case["own_max"] // page + 1
    pages = B * max_pages + F
    ids = shuffled(pages)
    order = shuffled(B)
    ended, sources = order[:F].contiguous(), order[F:F + case["sources"]]
    sources = sources[integers(0, case["sources"] - 1, F).long()].contiguous()
    used = (lens + page - 1) // page
    table = _tables(used, max_pages, ids[:B * max_pages])
    # the first pages of the rows in front belong to several sequences already
    twin = torch.arange(B, device="cuda") // 4 * 4
    both = (lens >= page) & (lens[twin] >= page)
    shared = torch.where(both, table[twin, 0], table[:, 0])
    table = torch.cat([shared[:, None], table[:, 1:]], 1)
    owners = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    owners.index_add_(0, torch.where(table >= 0, table, pages).reshape(-1).long(),
                      torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
    is_free = owners[:pages] == 0
    stack = torch.sort(torch.where(is_free, torch.arange(pages, device="cuda"), -1), descending=True).values
    flat, shapes = _index([table, lens, (owners[:pages] - 1).clamp(min=0), stack, is_free.sum().reshape(1)])
    pools = _pool_words(case, pages)
    return {"case": case, "start": flat, "shapes": shapes, "now": flat.clone(), "ended": ended, "sources": sources,
            "pools": pools, "each": list(pools.unbind(0))}


def _prepare_compact(case, normal, integers, shuffled):
    B, pages, live = case["B"], case["pages"], case["live"]
    ids = shuffled(pages)
    prefix = min(case["prefix"], live - 1)
    own_pages = live - prefix
    max_pages = -(-own_pages // B) + 1
    # the sequences' pages in turn, a third of them in a second row too
    rank = torch.arange(B * max_pages, device="cuda").reshape(max_pages, B).T
    table = torch.where(rank < own_pages, ids[prefix:live][rank.clamp(max=own_pages - 1)], -1)
    table = torch.cat([table, torch.where(rank[:, :1] % 3 == 0, table[:, :1], -1).roll(1, 0)], 1)
    owners = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    owners.index_add_(0, torch.where(table >= 0, table, pages).reshape(-1).long(),
                      torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
    shares = (owners[:pages] - 1).clamp(min=0)
    stack = torch.cat([ids[live:], torch.full((live,), -1, dtype=torch.int32, device="cuda")])
    flat, shapes = _index([table, ids[:prefix], shares, stack, torch.tensor([pages - live], device="cuda")])
    pools = _pool_words(case, pages)
    return {"case": case, "start": flat, "shapes": shapes, "now": flat.clone(), "pools": pools,
            "each": list(pools.unbind(0))}


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _own_attn, "append": _own_append, "linear": _own_linear, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"attn": _plain_attn, "append": _plain_append, "linear": _plain_linear, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


def _own_attn(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    B, K, hq, hkv, d = (c[k] for k in ("B", "K", "hq", "hkv", "d"))
    if "ws" not in s:  # a program keeps its workspace and its buffers
        s["ws"] = torch.zeros(sb.sv_kv4_attention_workspace_size(B, K, hq, hkv, d), dtype=torch.uint8, device="cuda")
        # rows behind a sequence's last draft stay as they are
        s["out"] = torch.zeros(B, K + 1, hq, d, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(B, K + 1, hq, device="cuda")
    sb.sv_kv4_attention(s["q"], 0, 0, 0, s["pool"], s["pool"].shape[0], c["page"], s["table"], s["table"].shape[1],
                        s["lens"], s["k"], c["window"], c["sinks"], s["scale"], s["out"], 0, 0, 0, s["lse"], BF16, B,
                        K, hq, hkv, d, s["ws"], s["ws"].numel())
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    B, T, hkv, d = (c[k] for k in ("B", "T", "hkv", "d"))
    if "ws" not in s:
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    kv, pool, table, out = s["kv"], s["pool"], s["table"], s["out"]
    row = 2 * hkv * d
    sb.sv_kv4_append(kv, kv.data_ptr() + hkv * d * 2, T * row, row, d, BF16, pool, pool.shape[0], c["page"], table,
                     table.shape[1], s["starts"], s["n"], B, T, hkv, d, s["ws"], 256)
    sb.sv_kv4_read(pool, pool.shape[0], c["page"], table, table.shape[1], s["starts"], s["n"], out[0], out[1], 0, 0, 0,
                   BF16, B, T, hkv, d, s["ws"], 256)
    return out


def _own_linear(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    M, N, K = c["M"], c["N"], c["K"]
    if "ws" not in s:
        s["ws"] = torch.zeros(sb.sv_linear_w4_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, dtype=TYPES[c["out"]], device="cuda")
    sb.sv_linear_w4(s["x"], 0, s["W"], 0, s["scales"], s["zeros"], c["group"], s["bias"], s["res"], 0, c["act"], out,
                    0, CODES[c["out"]], M, N, K, s["ws"], s["ws"].numel())
    return out


def _own_fork(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    F, pages = c["F"], s["pools"].shape[1]
    s["now"].copy_(s["start"])
    table, lens, shares, stack, top = _views(s["now"], s["shapes"])
    if "ws" not in s:
        s["ws"] = torch.zeros(sb.sv_kv_pages_workspace_size(pages, F), dtype=torch.uint8, device="cuda")
    ws = s["ws"]
    sb.sv_kv_free(table, table.shape[1], lens, shares, pages, stack, top, pages, s["ended"], F, c["B"], ws, ws.numel())
    sb.sv_kv_fork(s["each"], [c["page_bytes"]] * c["pools"], c["pools"], pages, c["page"], table, table.shape[1], lens,
                  shares, stack, top, s["sources"], s["ended"], F, c["B"], ws, ws.numel())
    return [table, lens, shares, torch.where(torch.arange(pages, device="cuda") < top, stack, -1), top, s["pools"]]


def _own_compact(s):
    from speculative_decoding_verification_47_gb300 import binding as sb
    c = s["case"]
    pages = c["pages"]
    s["now"].copy_(s["start"])
    table, prefix, shares, stack, top = _views(s["now"], s["shapes"])
    if "ws" not in s:
        s["ws"] = torch.zeros(sb.sv_kv_pages_workspace_size(pages, 0), dtype=torch.uint8, device="cuda")
    ws = s["ws"]
    sb.sv_kv_compact(s["each"], [c["page_bytes"]] * c["pools"], c["pools"], pages, table, table.shape[1], c["B"],
                     prefix if prefix.numel() else None, prefix.numel(), shares, stack, top, pages, ws, ws.numel())
    return [table, prefix, shares, torch.where(torch.arange(pages, device="cuda") < top, stack, -1), top, s["pools"]]


def _plain_attn(s):
    c = s["case"]
    B, K, hq, hkv, d, page = (c[k] for k in ("B", "K", "hq", "hkv", "d", "page"))
    G, Q = hq // hkv, K + 1
    ids = s["table"].long().clamp(min=0)                                # pages past a sequence's end are masked
    kv = _unpack(s["pool"][ids.reshape(-1)], hkv, d, page, torch.float32)
    kv = kv.reshape(2, B, ids.shape[1], hkv, page, d).transpose(2, 3).reshape(2, B, hkv, -1, d)
    q = s["q"].float().reshape(B, Q, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, Q * G, d) * s["scale"]
    z = q @ kv[0].transpose(2, 3)                                       # B hkv Q*G T
    i = torch.arange(Q, device="cuda")
    t = torch.arange(z.shape[3], device="cuda")
    at = (s["lens"][:, None] + i - 1)[..., None]                        # B Q 1
    seen = (t <= at) & ((t < c["sinks"]) | (t > at - c["window"])) if c["window"] else t <= at
    z = z.masked_fill(~seen.repeat_interleave(G, 1)[:, None], float("-inf"))
    m = z.amax(3, keepdim=True)
    ref = torch.where(torch.isfinite(m), m, 0.0)
    w = (z - ref).exp_()
    total = w.sum(3, keepdim=True)
    o = torch.where(total > 0, (w @ kv[1]) / total, 0.0)
    lse = (total.log() + ref)[..., 0]
    valid = i[None] <= s["k"][:, None]                                  # rows past k_b are not computed
    o = o.reshape(B, hkv, Q, G, d).transpose(1, 2).reshape(B, Q, hq, d)
    lse = lse.reshape(B, hkv, Q, G).transpose(1, 2).reshape(B, Q, hq)
    return {"out": torch.where(valid[..., None, None], o, 0.0).to(torch.bfloat16),
            "lse": torch.where(valid[..., None], lse, 0.0)}


def _plain_append(s):
    c = s["case"]
    B, T, hkv, d, page = (c[k] for k in ("B", "T", "hkv", "d", "page"))
    codes, scale, low = _quantise(s["kv"])                              # B T 2 hkv d
    i = torch.arange(T, device="cuda")
    at = s["starts"].long()[:, None] + i
    valid = (i[None] < s["n"][:, None]).reshape(-1)
    entry = torch.take_along_dim(s["table"].long(), at // page, 1).clamp(min=0)
    # a token's bytes in its page, for each head: codes of K and of V, and their (scale, minimum)
    head = (torch.arange(hkv, device="cuda") * _head_bytes(d, page))[None, None]
    base = entry[..., None] * s["pool"].shape[1] + head                 # B T hkv
    tok = (at % page)[..., None]
    nib = (codes[..., 0::2] | (codes[..., 1::2] << 4)).transpose(2, 3)  # B T hkv 2 d/2
    words = torch.stack([scale, low], -1).transpose(2, 3).contiguous().view(torch.uint8).reshape(B, T, hkv, 2, 4)
    half = torch.arange(2, device="cuda")[:, None]
    where = (base + tok * (d // 2))[..., None, None] + half * (page * d // 2) + torch.arange(d // 2, device="cuda")
    wordat = (base + page * d + tok * 4)[..., None, None] + half * (page * 4) + torch.arange(4, device="cuda")
    flat = s["pool"].view(-1)
    at_all = torch.cat([where.reshape(B * T, -1), wordat.reshape(B * T, -1)], 1)
    new = torch.cat([nib.reshape(B * T, -1), words.reshape(B * T, -1)], 1)
    # tokens past n stay as they are: their place is one behind the pool
    store = torch.cat([flat, flat.new_zeros(1)])
    store[torch.where(valid[:, None], at_all, flat.numel())] = new
    flat.copy_(store[:-1])
    got, words = flat[where], flat[wordat].contiguous().view(torch.bfloat16).float()
    values = torch.stack([got & 15, got >> 4], -1).reshape(B, T, hkv, 2, d).float()
    values = (words[..., 1:] + words[..., :1] * values).permute(3, 0, 1, 2, 4)
    return torch.where(valid.reshape(1, B, T, 1, 1), values, 0.0).to(torch.bfloat16)


def _activate(z, act):
    if act == RELU:
        return z.clamp(min=0)
    if act == SILU:
        return z / (1 + torch.exp(-z))
    if act == GELU:
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == GELU_TANH:
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def _weights(s, dtype):
    c = s["case"]
    codes = torch.stack([s["W"] & 15, s["W"] >> 4], -1).reshape(c["N"], -1, c["group"]).to(dtype)
    zeros = 8.0 if s["zeros"] is None else s["zeros"].to(dtype)[..., None]
    return ((codes - zeros) * s["scales"].to(dtype)[..., None]).reshape(c["N"], c["K"])


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ _weights(s, torch.float32).T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _activate(z, c["act"])
    if s["res"] is not None:
        z = z + s["res"].float()
    return z.to(TYPES[c["out"]])


def _plain_fork(s):
    c = s["case"]
    F, page, pages = c["F"], c["page"], s["pools"].shape[1]
    s["now"].copy_(s["start"])
    table, lens, shares, stack, top = _views(s["now"], s["shapes"])
    ended, sources = s["ended"].long(), s["sources"].long()
    every = torch.arange(pages, device="cuda")
    # the ended rows' pages lose an owner; those without one go on the stack, the lowest last
    rows = table[ended]
    gone = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    gone.index_add_(0, torch.where(rows >= 0, rows, pages).reshape(-1).long(), torch.ones_like(rows).reshape(-1))
    gone = gone[:pages]
    released = gone > shares
    shares.copy_(torch.where(released, 0, shares - gone))
    ids = torch.sort(torch.where(released, every, -1), descending=True).values
    n = released.sum().to(torch.int32)
    place = every - top
    stack.copy_(torch.where((place >= 0) & (place < n), ids[place.clamp(0, pages - 1)].to(torch.int32), stack))
    top += n
    table[ended] = -1
    lens[ended] = 0
    # the sources' whole pages get another owner, a page that is partly full is copied to one from the stack
    length = lens[sources]
    full, part = length // page, length % page > 0
    rank = torch.cumsum(part, 0) - part.long()
    fresh = stack[(top - 1 - rank).clamp(0, pages - 1).long()]
    rows = table[sources]
    j = torch.arange(table.shape[1], device="cuda")[None]
    shared = j < full[:, None]
    table[ended] = torch.where(shared, rows, torch.where((j == full[:, None]) & part[:, None], fresh[:, None], -1))
    more = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    more.index_add_(0, torch.where(shared, rows, pages).reshape(-1).long(), torch.ones_like(rows).reshape(-1))
    shares += more[:pages]
    lens[ended] = length
    last = torch.take_along_dim(rows, full[:, None].long().clamp(max=rows.shape[1] - 1), 1)[:, 0].clamp(min=0)
    # a fork without such a page copies the first one's again (a page onto itself if there is none)
    first = part.int().argmax()
    src = torch.where(part, last, last[first]).long()
    dst = torch.where(part, fresh, torch.where(part.any(), fresh[first], src)).long()
    s["pools"].index_copy_(1, dst, s["pools"][:, src])
    top -= part.sum().to(torch.int32)
    return [table, lens, shares, torch.where(every < top, stack, -1), top, s["pools"]]


def _plain_compact(s):
    c = s["case"]
    pages = c["pages"]
    s["now"].copy_(s["start"])
    table, prefix, shares, stack, top = _views(s["now"], s["shapes"])
    every = torch.arange(pages, device="cuda")
    used = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    used[torch.where(table >= 0, table, pages).reshape(-1).long()] = 1
    used[prefix.long()] = 1
    used = used[:pages] > 0
    live = used.sum()
    # the live pages behind the first `live`, and the free ones among these, in order
    most = pages // 2
    moves = torch.sort(torch.where(used & (every >= live), every, pages)).values[:most]
    holes = torch.sort(torch.where(~used & (every < live), every, pages)).values[:most]
    moved = moves < pages
    to = torch.cat([every, every[:1]]).to(torch.int32)
    to[moves] = torch.where(moved, holes, 0).to(torch.int32)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    prefix.copy_(to[prefix.long()])
    got = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    got[:pages] = torch.where(used & (every < live), shares, 0)
    got[torch.where(moved, holes, pages)] = torch.where(moved, shares[moves.clamp(max=pages - 1)], 0)
    shares.copy_(got[:pages])
    # (moves that are none copy the last page onto itself)
    src, dst = torch.where(moved, moves, pages - 1), torch.where(moved, holes, pages - 1)
    s["pools"].index_copy_(1, dst, s["pools"][:, src])
    top.copy_((pages - live).reshape(1))
    stack.copy_(torch.where(every < top, pages - 1 - every, stack))
    return [table, prefix, shares, torch.where(every < top, stack, -1), top, s["pools"]]


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "attn":
        # lengths and draft counts at their mean over prepare()'s draws
        k = (c["kmin"] + c["K"]) / 2
        n = (c["own_min"] + c["own_max"]) / 2
        seen = min(n, c["window"] + c["sinks"]) if c["window"] else n
        rows = c["B"] * (k + 1) * c["hq"]
        return {"bytes": c["B"] * (seen + k) * c["hkv"] * (c["d"] + 8) + rows * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * rows * (seen + (0 if c["window"] else k / 2))}
    if c["op"] == "append":
        values = c["B"] * (c["nmin"] + c["T"]) / 2 * c["hkv"] * c["d"] * 2
        return {"bytes": values * (2 + 2) + values * (c["d"] + 8) / (2 * c["d"]), "flops": 8 * values}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        e = 4 if c["out"] == "f32" else 2
        return {"bytes": N * K // 2 + N * K // c["group"] * (3 if c["zeros"] else 2) + M * K * 2
                + M * N * e * (2 if c["res"] else 1) + (N * 2 if c["bias"] else 0), "flops": 2 * M * N * K}
    if c["op"] == "fork":
        entries = (c["own_min"] + c["own_max"]) / 2 / c["page"] + 1
        copies = c["F"] * (1 - 1 / c["page"])
        return {"bytes": 2 * copies * c["pools"] * c["page_bytes"] + 24 * c["F"] * entries,
                "flops": c["F"] * entries}
    moves = c["live"] * (c["pages"] - c["live"]) / c["pages"]
    return {"bytes": 2 * moves * c["pools"] * c["page_bytes"] + 8 * c["live"] + 12 * c["pages"], "flops": c["pages"]}


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    kind = {"attn": _exact_attn, "append": _exact_append, "linear": _exact_linear}.get(case["op"])
    return None if kind is None else kind(prepare(case, seed))  # (pages are moved, not computed)


def _exact_tokens(pool, pages, hkv, d, page, n):
    """Keys and values [n][hkv][d] of a sequence's first n tokens, from its pages' bytes."""
    raw = pool[pages.long()].reshape(len(pages), hkv, -1)
    found = []
    for part in range(2):
        at = part * page * d // 2
        c = raw[:, :, at:at + page * d // 2].reshape(-1, hkv, page, d // 2).long()
        at = page * d + part * page * 4
        w = raw[:, :, at:at + page * 4].reshape(-1, hkv, page, 4).long()
        scale = ((w[..., 0] | w[..., 1] << 8) << 16).to(torch.int32).view(torch.float32).double()
        low = ((w[..., 2] | w[..., 3] << 8) << 16).to(torch.int32).view(torch.float32).double()
        values = torch.zeros(len(pages), hkv, page, d, dtype=torch.float64, device="cuda")
        values[..., 0::2], values[..., 1::2] = (c % 16).double(), (c // 16).double()
        values = values * scale[..., None] + low[..., None]
        found.append(values.transpose(1, 2).reshape(-1, hkv, d)[:n])
    return found


def _exact_attn(s):
    """Sequence by sequence and position by position: a softmax over exactly the keys it sees."""
    c = s["case"]
    B, K, hq, hkv, d, page = (c[k] for k in ("B", "K", "hq", "hkv", "d", "page"))
    G = hq // hkv
    lens, k = s["lens"].tolist(), s["k"].tolist()
    out = torch.zeros(B, K + 1, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, K + 1, hq, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = lens[b] + k[b]
        if n == 0:
            lse[b, 0] = -math.inf
            continue
        keys, values = _exact_tokens(s["pool"], s["table"][b, :-(-n // page)], hkv, d, page, n)
        q = s["q"][b].double().reshape(K + 1, hkv, G, d)
        for i in range(k[b] + 1):
            end = lens[b] + i
            at = list(range(0, min(c["sinks"], end))) if c["window"] else []
            begin = max(len(at), end - c["window"]) if c["window"] else 0
            if end == 0:
                lse[b, i] = -math.inf
                continue
            ks, vs = (torch.cat([a[:len(at)], a[begin:end]]) for a in (keys, values))
            z = torch.einsum("hgd,nhd->hgn", q[i], ks) * s["scale"]
            lse[b, i] = torch.logsumexp(z, 2).reshape(hq)
            out[b, i] = torch.einsum("hgn,nhd->hgd", torch.softmax(z, 2), vs).reshape(hq, d)
    return {"out": out, "lse": lse}


def _exact_bf16(v):
    """The nearest values of 8 significant bits, ties to even: 45 of the 52 bits behind the leading one go."""
    bits = v.contiguous().view(torch.int64)
    bits = bits + ((1 << 44) - 1) + ((bits >> 45) & 1)
    return ((bits >> 45) << 45).view(torch.float64)


def _exact_append(s):
    c = s["case"]
    x = s["kv"].double().permute(2, 0, 1, 3, 4)                         # 2 B T hkv d
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    scale = _exact_bf16(torch.div(high - low, torch.full_like(low, 15)))
    codes = torch.clamp(torch.round((x - low) / torch.where(scale > 0, scale, 1.0)), 0, 15)
    valid = torch.arange(c["T"], device="cuda")[None] < s["n"][:, None]
    return torch.where(valid[None, :, :, None, None], low + torch.where(scale > 0, codes, 0.0) * scale, 0.0)


def _exact_linear(s):
    c = s["case"]
    W = torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
    W[:, 0::2], W[:, 1::2] = (s["W"] % 16).double(), (s["W"] // 16).double()
    W = W.reshape(c["N"], -1, c["group"])
    W = W - (8.0 if s["zeros"] is None else s["zeros"].double()[..., None])
    z = torch.einsum("mgk,ngk->mn", s["x"].double().reshape(c["M"], -1, c["group"]), W * s["scales"].double()[..., None])
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
