"""Rounds of a decode over one paged cache: each writes the emitted token's keys and values at
the committed length and passes that length plus one, so that every query sees its own token;
attention, commit and the pages that the commit gives back follow one another.  Each sequence's
tokens are kept apart as a plain list, and each round's outputs are those of a softmax over it."""

import numpy as np
import pytest

from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


@pytest.mark.parametrize("page", [4, 16])
def test_rounds_see_their_own_tokens(page):
    r = np.random.default_rng(page)
    g = torch.Generator().manual_seed(page)
    B, K, hq, hkv, D, P, max_pages = 6, 3, 4, 2, 64, 10, 64 // page
    num_pages = -(-P // page) + B * max_pages + 3
    normal = lambda *s: torch.randn(*s, generator=g).to(BF)
    kp, vp = (torch.full((num_pages, page, hkv, D), float("nan")).to(BF) for _ in range(2))
    free = r.permutation(num_pages).astype(np.int32).tolist()
    prefix = [free.pop() for _ in range(-(-P // page))]
    prefix_kv = [(normal(hkv, D), normal(hkv, D)) for _ in range(P)]
    table = np.full((B, max_pages), -1, np.int32)

    def write(pages, at, kv):
        kp[pages[at // page], at % page], vp[pages[at // page], at % page] = kv

    def append(b, at, kv):
        if table[b, at // page] < 0:
            table[b, at // page] = free.pop()
        write(table[b], at, kv)

    for j, kv in enumerate(prefix_kv):
        write(prefix, j, kv)
    tokens = [[(normal(hkv, D), normal(hkv, D)) for _ in range(int(n))] for n in r.integers(1, 12, B)]
    for b in range(B):
        for j, kv in enumerate(tokens[b]):
            append(b, j, kv)
    f64 = lambda kv, i: np.array([t[i].double().numpy() for t in kv]).reshape(-1, hkv, D)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    ws = torch.empty(sb.sv_prefix_attention_workspace_size(B, K, hq, hkv, D, P, max_pages * page), dtype=torch.uint8,
                     device="cuda")
    cws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dlens = dev(np.array([len(t) for t in tokens], np.int32))
    for _ in range(5):
        ks = r.integers(0, K + 1, B).astype(np.int32)
        drafts = [[(normal(hkv, D), normal(hkv, D)) for _ in range(int(k))] for k in ks]
        for b in range(B):
            for j, kv in enumerate(drafts[b]):
                append(b, len(tokens[b]) + j, kv)
        q = normal(B, K + 1, hq, D)
        out = torch.empty(B, K + 1, hq, D, dtype=BF, device="cuda")
        dtable = dev(table)
        sb.sv_prefix_attention(q.cuda(), 0, 0, 0, kp.cuda(), vp.cuda(), 0, 0, 0, num_pages, page,
                               dev(np.array(prefix, np.int32)), P, dtable, max_pages, dlens, dev(ks), D ** -0.5, out,
                               0, 0, 0, None, sb.SV_BF16, B, K, hq, hkv, D, ws, ws.numel())
        assert sb.sv_read_device_flags(ws) == 0
        for b in range(B):
            own, k = tokens[b] + drafts[b], int(ks[b])
            ref, _, weight, _ = oy.prefix_attention(q[b, :k + 1].double().numpy(), f64(prefix_kv, 0),
                                                    f64(prefix_kv, 1), f64(own, 0), f64(own, 1), len(tokens[b]),
                                                    D ** -0.5)
            # halves of a bf16 step of the weights and of the output, and float32's sums
            off = np.abs(out[b, :k + 1].double().cpu().numpy() - ref)
            assert np.all(off <= (2.0 ** -8 + 2.0 ** -14) * weight + 2.0 ** -8 * np.abs(ref))
        n = np.array([r.integers(0, k + 1) for k in ks], np.int32)
        stack = torch.full((num_pages,), -7, dtype=torch.int32, device="cuda")
        top = torch.zeros(1, dtype=torch.int32, device="cuda")
        sb.sv_kv_commit_paged(dlens, dev(n), dev(ks), dtable, max_pages, page, stack, top, num_pages, B, cws, 256)
        assert sb.sv_read_device_flags(cws) == 0
        free += stack[:int(top.item())].cpu().tolist()
        table = dtable.cpu().numpy()
        for b in range(B):
            tokens[b] += drafts[b][:n[b]]
            assert int(dlens[b]) == len(tokens[b])
            tokens[b].append((normal(hkv, D), normal(hkv, D)))  # the emitted token, which this round has not seen
            append(b, len(tokens[b]) - 1, tokens[b][-1])
        dlens += 1
