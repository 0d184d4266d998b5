"""The example that runs the decode-step operators together: every operator's output in a
step against 64 bits from that step's own inputs, and a captured step replayed against eager
steps bit for bit."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

_spec = importlib.util.spec_from_file_location(
    "decode_block", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                 "examples", "decode_block.py"))
ex = importlib.util.module_from_spec(_spec)
import sys  # noqa: E402

sys.modules["decode_block"] = ex
_spec.loader.exec_module(ex)


def session(fp8, B=5, P=83, new=12):
    cfg = ex.Config(fp8_cache=fp8)
    block = ex.Block(cfg)
    prompt = torch.randint(0, cfg.vocab, (P,), generator=torch.Generator().manual_seed(1))
    s = ex.Session(block, prompt, B, new)
    s.token.copy_(torch.arange(B, device="cuda:0", dtype=torch.int32) * 11 + 3)
    return s


def dequant(w):
    q, scale, zero = (t.cpu() if t is not None else None for t in w._keep)
    fmt = "fp4" if w.format == moe.MOE_W_FP4_E2M1_UE8M0_K32 else "int4"
    return ref.w4_dequant(fmt, q.numpy(), scale.numpy() if fmt == "fp4" else scale,
                          zero.numpy() if zero is not None else None, w.group)[0]


@pytest.mark.parametrize("fp8", [False, True])
def test_a_step_against_64_bits(fp8):
    s = session(fp8)
    c, b = s.cfg, s.block
    for i in range(3):
        tok, pos = s.token.clone(), s.pos.cpu().numpy()
        s.step()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
    x = ex.rms_norm(b.embed[tok]).double().cpu().numpy()
    # bf16 outputs: half a unit is 2^-8 of the value; fp32 sums well below
    qkv = x @ dequant(b.qkv).T
    got = s.qkv.double().cpu().numpy()
    assert (np.abs(got - qkv) <= 2.0 ** -8 * np.abs(qkv) + 1e-5).all()
    # q rotated, k and v in their slots
    D, Hq, Hkv = c.head_dim, c.q_heads, c.kv_heads
    f = s.qkv.float().cpu().numpy().reshape(s.B, Hq + 2 * Hkv, D)
    r = ref.rotate_f32(f[:, :Hq + Hkv], s.rope.cpu().numpy()[pos], D, False)
    assert torch.equal(s.q.cpu(), ref.bf16(r[:, :Hq]))
    kv = ref.Cache.__new__(ref.Cache)
    kv.page, kv.fp8 = c.page, fp8
    kv.t = {"k": s.k.cpu(), "v": s.v.cpu(), "ks": s.ks.cpu() if fp8 else None,
            "vs": s.vs.cpu() if fp8 else None}
    K, V = kv.values("k"), kv.values("v")
    table = s.table.cpu().numpy()
    for bq in range(s.B):
        pg, sl = table[bq, pos[bq] // c.page], pos[bq] % c.page
        tol = 2.0 ** -4 if fp8 else 2.0 ** -8
        for new, buf in ((r[bq, Hq:], K), (f[bq, Hq + Hkv:], V)):
            # E4M3: half a unit is 2^-4 of the value, below the least normal 2^-10 of the scale
            sc = np.abs(new).max(-1, keepdims=True) / 448 * 2.0 ** -10 if fp8 else 0
            assert (np.abs(buf[pg, :, sl] - new) <= 1.001 * tol * np.abs(new) + sc).all()
    # attention, output projection, log probabilities, each from its own inputs
    eo, el, mag, _ = ref.attention(s.q.double().cpu().numpy(), kv, pos, s.prefix_pages.tolist(), s.P,
                                   table, D ** -0.5, 1, s.max_keys)
    o = s.att.double().cpu().numpy()
    assert (np.abs(o - eo) <= 1.05 * 2.0 ** -8 * (mag + np.abs(eo)) + 2.0 ** -12 * mag).all()
    assert np.abs(s.lse.double().cpu().numpy() - el).max() <= 1e-4
    proj = o.reshape(s.B, -1) @ dequant(b.out).T
    assert (np.abs(s.o.double().cpu().numpy() - proj) <= 2.0 ** -8 * np.abs(proj) + 1e-5).all()
    z = s.logits.double().cpu().numpy()
    lp = z - z.max(1, keepdims=True)
    lp -= np.log(np.exp(lp).sum(1, keepdims=True))
    order = np.argsort(-z, axis=1, kind="stable")[:, :c.alternatives]
    assert np.array_equal(s.top_ids.cpu().numpy(), order)
    assert np.abs(s.top_lp.cpu().numpy() - np.take_along_axis(lp, order, 1)).max() <= 1e-5
    assert np.abs(s.entropy.cpu().numpy() + (np.exp(lp) * lp).sum(1)).max() <= 1e-4
    assert torch.equal(s.token, s.top_ids[:, 0])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_captured_step_replays_as_eager_steps(fp8):
    eager, cap = session(fp8), session(fp8)
    for s in (eager, cap):
        s.step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st, capture_error_mode="relaxed"):
        cap.step()
    for i in range(5):
        eager.step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n in ("token", "pos", "logits", "top_ids", "top_lp", "entropy", "att", "k", "v"):
            assert torch.equal(getattr(eager, n), getattr(cap, n)), (i, n)
