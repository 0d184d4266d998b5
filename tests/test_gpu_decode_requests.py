"""The example's step for requests that differ (norms with residual and E4M3 output, adapters, a cache
in 4 bits, rules on logits): every operator's output against 64 bits from that step's own inputs, and
a captured step replayed against eager steps bit for bit."""
import numpy as np
import pytest
import torch

import dense_ref
import ops_ref as ref
from test_gpu_cache_fp4 import Cache4, fp4_rows
from test_gpu_decode_block import dequant, ex, moe

pytestmark = pytest.mark.gpu


def session(fp4, B=7, P=83, new=12):
    cfg = ex.Config(fp4_cache=fp4, requests=True)
    block = ex.Block(cfg)
    prompt = torch.randint(0, cfg.vocab, (P,), generator=torch.Generator().manual_seed(1))
    s = ex.Session(block, prompt, B, new)
    s.token.copy_(torch.arange(B, device="cuda:0", dtype=torch.int32) * 11 + 3)
    return s


def np64(t):
    return t.double().cpu().numpy()


def rms(r, w):
    return r / np.sqrt((r * r).mean(1, keepdims=True) + float(np.float32(1e-6))) * w


def near_bf16(got, want, more=0.0):
    """Half a unit of bf16 and 2^-18 of fp32 sums (test_gpu_add_rmsnorm), and what is said."""
    assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + more + 1e-30).all(), \
        np.abs(got - want).max()


@pytest.mark.parametrize("fp4", [False, True])
def test_a_step_against_64_bits(fp4):
    s = session(fp4)
    c, b = s.cfg, s.block
    for i in range(4):
        tok, pos, n_before = s.token.clone(), s.pos.cpu().numpy(), s.n_tokens.clone()
        kept = []
        norm = s._norm
        s._norm = lambda which, x, *a, **k: (norm(which, x, *a, **k), kept.append(np64(a[3]) if which < 2 else None))
        s.step()
        torch.cuda.synchronize()
        s._norm = norm
        assert int(s.status.item()) == 0
    w = np64(b.norms)
    e = np64(b.embed[tok])
    # q/k/v: the first norm, the shared projection (rounded to bf16), then the adapters on top (rounded
    # once more)
    x0 = kept[0]
    near_bf16(x0, rms(e, w[0]))
    base = x0 @ dequant(b.qkv).T
    a_, b_, rank, scale = (t.cpu() for t in b.qkv_lora._keep)
    delta, mag = np.zeros_like(base), np.zeros_like(base)
    for t, i in enumerate(s.adapter.tolist()):
        if i >= 0:
            A, Bm = np64(a_[i, :int(rank[i])]), np64(b_[i, :, :int(rank[i])])
            delta[t] = Bm @ (A @ x0[t]) * float(scale[i])
            mag[t] = np.abs(Bm) @ (np.abs(A) @ np.abs(x0[t])) * float(scale[i])
    got = np64(s.qkv)
    assert (np.abs(got - base - delta) <= 2.0 ** -8 * (np.abs(base) + np.abs(base + delta)) * 1.01 +
            2.0 ** -13 * mag + 1e-5).all()
    # the cache's rows of this step
    D, Hq, Hkv = c.head_dim, c.q_heads, c.kv_heads
    f = s.qkv.float().cpu().numpy().reshape(s.B, Hq + 2 * Hkv, D)
    r = ref.rotate_f32(f[:, :Hq + Hkv], s.rope.cpu().numpy()[pos], D, False)
    assert torch.equal(s.q.cpu(), ref.bf16(r[:, :Hq]))
    table = s.table.cpu().numpy()
    if fp4:
        kv = Cache4.__new__(Cache4)
        kv.page, kv.t = c.page, {n: getattr(s, n).cpu() for n in ("k", "v", "ks", "vs")}
        for bq in range(s.B):
            pg, sl = table[bq, pos[bq] // c.page], pos[bq] % c.page
            for n, new in (("k", r[bq, Hq:]), ("v", f[bq, Hq + Hkv:])):
                codes, sb = fp4_rows(new)
                assert np.array_equal(kv.t[n][pg, :, sl].numpy(), codes)
                assert np.array_equal(kv.t[n + "s"][pg, :, sl].numpy(), sb)
    else:
        kv = ref.Cache.__new__(ref.Cache)
        kv.page, kv.fp8, kv.t = c.page, False, {"k": s.k.cpu(), "v": s.v.cpu(), "ks": None, "vs": None}
    eo, el, m, _ = ref.attention(np64(s.q), kv, pos, s.prefix_pages.tolist(), s.P, table, D ** -0.5, 1,
                                 s.max_keys)
    o = np64(s.att)
    assert (np.abs(o - eo) <= 1.05 * 2.0 ** -8 * (m + np.abs(eo)) + 2.0 ** -12 * m).all()
    # residual, norm and E4M3 activations; the experts from exactly these
    stream = (b.embed[tok].float() + s.o.float()).to(torch.bfloat16)
    assert torch.equal(s.stream, stream)
    y = rms(np64(stream), w[1])
    near_bf16(np64(s.mid), y)
    xd = np64(s.xq.view(torch.float8_e4m3fn)) * np.repeat(np64(s.xs), 128, 1)
    assert (np.abs(xd - y) <= 1.001 * (2.0 ** -4 * np.abs(y) + 2.0 ** -10 * np.repeat(np64(s.xs), 128, 1))).all()
    E = [t.cpu().numpy() for t in b.moe._keep]
    mats = {}

    def ffn(i, x):
        if i not in mats:
            mats[i] = [dense_ref.dense_fp4(E[2 * j][i], E[2 * j + 1][i]) for j in range(3)]
        G, U, Dn = mats[i]
        g, u = x @ G.T, x @ U.T
        hq, hs = dense_ref.quant_torch((g / (1 + np.exp(-g)) * u).astype(np.float32)[None])
        return (dense_ref.dequant_act(hq, hs) @ Dn.T)[0]
    want = np.stack([ffn(c.experts, xd[t]) + sum(float(s.gate[t, j]) * ffn(int(s.ids[t, j]), xd[t])
                                                 for j in range(c.top_k)) for t in range(s.B)])
    got = np64(s.ffn)
    # (the layer's own parity bound, and half a unit of bf16)
    assert np.linalg.norm(got - want) <= (2e-3 + 2.0 ** -8) * np.linalg.norm(want)
    last = (s.ffn.float() + s.stream.float()).to(torch.bfloat16)
    near_bf16(np64(s.xn), rms(np64(last), w[2]))
    # rules: the text so far, with this step's token
    n = n_before.tolist()
    for t in range(s.B):
        assert int(s.text[t, n[t]]) == int(tok[t])
    z = np64(s.logits)
    k = s.rules._keep
    rep, pres, freq = np64(k[4]), np64(k[5]), np64(k[6])
    for t in range(s.B):
        e = z[t].copy()
        e[s.bias_ids[t].cpu().numpy()] += np64(s.bias[t])
        text = s.text[t, :n[t] + 1].cpu().numpy()
        met = np.unique(text)
        e[met] = np.where(e[met] > 0, e[met] / rep[t], e[met] * rep[t])
        ids, cnt = np.unique(text[s.P:], return_counts=True)
        e[ids] -= pres[t] + freq[t] * cnt
        if int(s.mask_of[t]) >= 0:
            e[1::2] = -np.inf
        got = np64(s.ruled[t])
        assert np.array_equal(np.isinf(got), np.isinf(e))
        with np.errstate(invalid="ignore"):
            assert (np.abs(got - e) <= 8 * 2.0 ** -24 * (np.abs(z[t]) + 4 + np.abs(e)))[np.isfinite(e)].all()
        order = np.argsort(-got, kind="stable")[:c.alternatives]
        assert np.array_equal(s.top_ids[t].cpu().numpy(), order)
    assert torch.equal(s.token, s.top_ids[:, 0])


@pytest.mark.parametrize("fp4", [False, True])
def test_a_captured_step_replays_as_eager_steps(fp4):
    eager, cap = session(fp4), session(fp4)
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
        for n in ("token", "pos", "logits", "ruled", "text", "n_tokens", "top_ids", "top_lp", "entropy", "att",
                  "xq", "xs", "ffn", "k", "v"):
            assert torch.equal(getattr(eager, n), getattr(cap, n)), (i, n)
    assert int(cap.status.item()) == 0


def test_steps_past_the_last_new_token_are_refused_by_the_status():
    """The text is full after `new` tokens: a further step stays inside it and says so."""
    s = session(True, B=3, P=20, new=2)
    for _ in range(2):
        s.step()
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    text = s.text.clone()
    for _ in range(2):
        s.step()
    torch.cuda.synchronize()
    assert int(s.status.item()) == moe.MOE_STATUS_BAD_PAGE | moe.MOE_STATUS_BAD_INDEX
    assert torch.equal(s.text[:, :-1], text[:, :-1])
