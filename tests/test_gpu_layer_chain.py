"""One layer of a target's forward over a round's positions and the step that judges
them, chained on the GPU: attention over the shared prefix and the paged cache, its
projection, the residual norm with an 8-bit output, an 8-bit feed-forward product
with its activation, the product back onto the residual stream, the LM head, the
verify step and the commit that rolls the paged cache back.  Every stage is checked
against its oracle fed with the GPU's own results of the stage before."""

import numpy as np
import pytest

from oracle import layer as oy
from oracle import lmhead as ol
from oracle import paged as opg
from speculative_decoding_verification_47_gb300 import binding as sb
from speculative_decoding_verification_47_gb300 import workloads as wl
from tests import verify_harness as vh
from tests.conftest import gpu_available
from tests.test_gpu_attention import Case

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def f64(t):
    return t.double().cpu().numpy()


def linear(x, W, M, N, K, ws, sx=None, sw=None, res=None, act=0):
    code = sb.SV_BF16 if x.dtype == BF else sb.SV_E4M3
    out = torch.empty(M, N, dtype=BF, device="cuda")
    sb.sv_linear(x, 0, sx, W, 0, sw, code, None, res, 0, act, out, 0, sb.SV_BF16, M, N, K, ws, ws.numel())
    ref, absp = oy.linear(f64(x), f64(W), None if sx is None else f64(sx), None if sw is None else f64(sw), None, act,
                          None if res is None else f64(res))
    # K float32 additions of exact products, the activation, half a bf16 step
    bound = 1.13 * (K + 8) * 2.0 ** -23 * absp + 2.0 ** -18 * (absp + 4) * (act != 0) + 2.0 ** -21 * (absp + 4)
    bound = bound + (2.0 ** -8 + 2.0 ** -23) * (np.abs(ref) + bound)
    assert np.all(np.abs(f64(out) - ref) <= bound)
    return out


def test_layer_then_verify_then_commit():
    r = np.random.default_rng(17)
    B, K, hq, hkv, D, F, V, page = 12, 4, 8, 2, 64, 1024, 4112, 16
    H, M = hq * D, B * (K + 1)
    lens, ks = r.integers(20, 120, B), r.integers(0, K + 1, B)
    c = Case(lens, ks, K, hq=hq, hkv=hkv, D=D, page=page, prefix=150, seed=7, max_pages=9)
    c.q = torch.nan_to_num(c.q)
    c.upload()
    c.run().check()
    attn = torch.where(c.out == 55.0, 0, c.out).reshape(M, H).to(BF)  # positions past k_b stayed as they were

    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF)
    ws = torch.zeros(sb.sv_linear_workspace_size(M, F, H), dtype=torch.uint8, device="cuda")
    stream = normal(M, H, scale=2.0)
    proj = linear(attn, normal(H, H, scale=H ** -0.5), M, H, H, ws)

    # the sum goes into the residual stream's own place, the normalised rows out in 8 bits
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF)
    before = f64(stream)
    y8 = torch.empty(M, H, dtype=torch.float8_e4m3fn, device="cuda")
    sx = torch.empty(M, device="cuda")
    sb.sv_rmsnorm_residual(proj, 0, stream, 0, w, 1e-5, stream, 0, sb.SV_BF16, y8, 0, sb.SV_E4M3, sx, M, H)
    s, y = oy.rmsnorm_residual(f64(proj), before, f64(w), 1e-5)
    assert np.all(np.abs(f64(stream) - s) <= 2.0 ** -8 * np.abs(s))
    assert np.all(np.abs(f64(sx) - oy.row_scale(y)) <= 2.0 ** -16 * oy.row_scale(y))
    # half an e4m3 step: 2^-4 of the value, or 2^-10 of the scale where the step is the smallest one
    off = np.abs(f64(y8) * f64(sx)[:, None] - y)
    assert np.all(off <= np.maximum((2.0 ** -4 + 2.0 ** -14) * np.abs(y), 2.0 ** -10 * 1.001 * f64(sx)[:, None]))

    Wu = torch.randn(F, H, generator=g, device="cuda") * H ** -0.5
    sw = Wu.abs().amax(1) / 448
    W8 = (Wu / sw[:, None]).to(torch.float8_e4m3fn)
    up = linear(y8, W8, M, F, H, ws, sx, sw, act=sb.SV_ACT_SILU)
    hidden = linear(up, normal(H, F, scale=F ** -0.5), M, H, F, ws, res=stream)
    assert sb.sv_read_device_flags(ws) == 0

    nw, Wv = normal(H, scale=0.1) + 1, normal(H, V, scale=0.05)
    logits = torch.empty(M, V, dtype=BF, device="cuda")
    lws = torch.zeros(sb.sv_lmhead_workspace_size(M, H), dtype=torch.uint8, device="cuda")
    sb.sv_lmhead_rmsnorm(hidden, nw, 1e-5, Wv, logits, sb.SV_BF16, M, H, V, lws, lws.numel())
    assert sb.sv_read_device_flags(lws) == 0
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)
    ref = ol.lmhead_rmsnorm(bits(hidden), bits(nw), 1e-5, bits(Wv))
    bound = 2.0 ** -7 * ol.lmhead_abs_product(bits(hidden), bits(nw), 1e-5, bits(Wv)) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(f64(logits) - ref) <= bound)

    target = bits(logits).reshape(B, K + 1, V)
    draft = wl.f64_to_bf16_bits(wl.bf16_bits_to_f32(target[:, :K]).astype(np.float64) + 0.5 * r.standard_normal((B, K, V)))
    kpr = c.ks.astype(np.int32)
    ones, mode = np.ones(B, np.float32), np.zeros(B, np.uint8)
    tokens = wl.draw_draft_tokens(draft, wl.BF16, kpr, ones, mode, seed=5)
    u = (r.integers(0, 1 << 24, size=(B, K + 1)) * 2.0 ** -24).astype(np.float32)
    v = wl.VerifyInputs(name="layer", dtype=wl.BF16, B=B, K=K, V=V, target=target, draft=draft, draft_tokens=tokens,
                        k_per_row=kpr, temperature=ones, top_p=1.0, uniforms=u, mode=mode, sigma=np.zeros(B))
    got = vh.run_gpu(v)
    vh.compare(v, got, vh.run_oracle(v))

    # the tables that attention read are the ones that the commit rolls back
    n = got.n.astype(np.int32)
    table = np.where(c.table < 10 ** 8, c.table, -1).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    dl, dt = dev(c.lens), dev(table)
    free = torch.full((c.num_pages,), -7, dtype=torch.int32, device="cuda")
    top = torch.zeros(1, dtype=torch.int32, device="cuda")
    cws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sb.sv_kv_commit_paged(dl, dev(n), dev(kpr), dt, c.max_pages, page, free, top, c.num_pages, B, cws, 256)
    rl, rt, rr, rtop, rflags = opg.kv_commit_paged(c.lens, n, kpr, table, page, 0, c.num_pages)
    assert sb.sv_read_device_flags(cws) == rflags == 0
    assert np.array_equal(dl.cpu().numpy(), rl) and np.array_equal(dt.cpu().numpy(), rt)
    assert int(top.item()) == rtop and sorted(free.cpu().numpy()[:rtop].tolist()) == sorted(rr)

    # the next round's attention over the rolled-back lengths and tables
    c.lens, c.table, c.ks = np.array(rl, np.int32), np.array(rt, np.int32), np.zeros(B, np.int32)
    c.upload()
    c.run().check()
