"""What is measured of the decode-step operators: 4-bit linears, the paged key/value cache with
its rotation, attention over a shared prefix, and token log probabilities.

Every case can be run in two forms on the same inputs: the plain form (elementary torch operations
in 32 bits, rounded once at the end) and, with `own` set, the library's operators.
"""
from __future__ import annotations

import math
import random

import torch

own = False
DEV = "cuda:0"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a hidden x hidden projection of the layer's model width: latency
        dict(name="linear_fp4_t1", op="linear", fmt="fp4", group=32, zeros=False, T=1, N=4096,
             K=4096, out="bf16"),
        # a ragged projection for five tokens: odd outputs, a last group cut short, zero points
        dict(name="linear_int4_t5_odd", op="linear", fmt="int4", group=128, zeros=True, T=5, N=1031,
             K=2080, out="f32"),
        # fused q/k/v projection (32 + 2 x 8 heads of 128) of a batch of 16 sequences
        dict(name="linear_int4_qkv_t16", op="linear", fmt="int4", group=128, zeros=True, T=16,
             N=6144, K=4096, out="bf16"),
        # vocabulary projection of a 32-token verification batch: the largest weight there is
        dict(name="linear_fp4_vocab_t32", op="linear", fmt="fp4", group=32, zeros=False, T=32,
             N=131072, K=4096, out="bf16"),
        # one decode step of 32 sequences: q rotated, k and v appended, bf16 cache
        dict(name="append_decode_b32", op="append", cache="bf16", T=32, B=32, Hq=32, Hkv=8, D=128,
             page=16, rot=128, style="half", past=1000),
        # an 8192-token prompt into an FP8 cache, half of each head rotated in interleaved pairs
        dict(name="append_prompt_fp8", op="append", cache="fp8", T=8192, B=1, Hq=32, Hkv=8, D=128,
             page=64, rot=64, style="pairs", past=0),
        # a small batch behind a short system prompt that ends inside a page: latency
        dict(name="attn_small_b4", op="attn", cache="bf16", B=4, Q=1, Hq=8, Hkv=2, D=64, page=16,
             prefix=500, own_max=60, pad=True),
        # ordinary decode: 32 sequences of up to 2048 tokens of their own behind 8192 shared ones
        dict(name="attn_decode_b32", op="attn", cache="bf16", B=32, Q=1, Hq=32, Hkv=8, D=128,
             page=64, prefix=8192, own_max=2048, pad=False),
        # speculative verification: 4 tokens for each of 16 sequences, a long shared document, FP8
        dict(name="attn_verify_fp8", op="attn", cache="fp8", B=16, Q=4, Hq=64, Hkv=8, D=128,
             page=64, prefix=32768, own_max=1024, pad=False),
        # one sampled token with its 20 best alternatives: latency
        dict(name="logprobs_t1_top20", op="logprobs", dtype="f32", T=1, V=131072, top=20),
        # a verification batch's tokens with 5 alternatives
        dict(name="logprobs_t32_top5", op="logprobs", dtype="bf16", T=32, V=131072, top=5),
        # scoring a prompt: every token's log probability and entropy, odd vocabulary
        dict(name="logprobs_prompt_t4096", op="logprobs", dtype="bf16", T=4096, V=50021, top=1),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    op = rng.choice(["linear", "linear", "append", "attn", "attn", "logprobs"])
    if op == "linear":
        fmt = rng.choice(["fp4", "int4"])
        T = _logu(rng, 1, 64)
        K = 32 * _logu(rng, 4, 256)
        N = _logu(rng, 64, max(65, min(131072, (131072 * 4096 * 32) // (K * max(T, 32)))))
        return dict(op=op, fmt=fmt, group=32 if fmt == "fp4" else rng.choice([32, 64, 128]),
                    zeros=fmt == "int4" and rng.random() < 0.5, T=T, N=N, K=K,
                    out=rng.choice(["bf16", "f32"]))
    if op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 128, 256])
        prompt = rng.random() < 0.5
        T = _logu(rng, 64, 4096) if prompt else _logu(rng, 1, 128)
        return dict(op=op, cache=rng.choice(["bf16", "fp8"]), T=T, B=1 if prompt else T,
                    Hq=Hkv * rng.choice([1, 3, 4]), Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]),
                    rot=rng.choice([D, D // 2]), style=rng.choice(["half", "pairs"]),
                    past=_logu(rng, 1, 2000))
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 7, 8])
        return dict(op=op, cache=rng.choice(["bf16", "fp8"]), B=_logu(rng, 1, 32),
                    Q=rng.choice([1, 1, 2, 4]), Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), prefix=_logu(rng, 16, 16384),
                    own_max=_logu(rng, 8, 1024), pad=rng.random() < 0.3)
    return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_logu(rng, 1, 1024),
                V=_logu(rng, 1000, 100000), top=rng.choice([0, 1, 5, 20]))


# ---------------------------------------------------------------- inputs

def _pages(n_keys, page):
    return -(-n_keys // page)


def _last(c):
    """Position of the last query of each sequence of an attention case: its own part between Q and
    own_max keys, spread over the batch; the last sequence of a padded batch is empty (-1)."""
    r = random.Random(c["B"] * 1000003 + c["own_max"])
    got = [c["prefix"] + c["Q"] - 1 + r.randrange(max(1, c["own_max"] - c["Q"] + 1))
           for _ in range(c["B"])]
    if c["pad"] and c["B"] > 1:
        got[-1] = -1
    return got


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": case, "op": case["op"]}
    {"linear": _prepare_linear, "append": _prepare_append, "attn": _prepare_attn,
     "logprobs": _prepare_logprobs}[case["op"]](case, g, s)
    if own:
        _handles(case, s)
    return s


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _bytes(g, *shape):
    return torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)


def _prepare_linear(c, g, s):
    T, N, K, G = c["T"], c["N"], c["K"], c["group"]
    n_g = -(-K // G)
    s["x"] = _normal(g, T, K).to(torch.bfloat16)
    s["q"] = _bytes(g, N, K // 2)
    if c["fmt"] == "fp4":      # scales 2^-8 .. 2^-4
        s["scale"] = torch.randint(119, 124, (N, n_g), generator=g, device=DEV, dtype=torch.uint8)
        s["zero"] = None
    else:
        s["scale"] = (0.002 + 0.01 * torch.rand((N, n_g), generator=g, device=DEV)).to(torch.bfloat16)
        s["zero"] = torch.randint(5, 12, (N, n_g), generator=g, device=DEV,
                                  dtype=torch.uint8) if c["zeros"] else None


def _cache(c, g, n_pages):
    shape = (n_pages, c["Hkv"], c["page"], c["D"])
    if c["cache"] == "bf16":
        return dict(k=_normal(g, *shape).to(torch.bfloat16), v=_normal(g, *shape).to(torch.bfloat16),
                    ks=None, vs=None)
    # FP8 pages as an append leaves them: the largest of a row is 448 times its scale
    k, v = _normal(g, *shape), _normal(g, *shape)
    ks, vs = k.abs().amax(-1) / 448.0, v.abs().amax(-1) / 448.0
    return dict(k=(k / ks[..., None]).to(torch.float8_e4m3fn), ks=ks,
                v=(v / vs[..., None]).to(torch.float8_e4m3fn), vs=vs)


def _rope_table(rows, rot):
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * \
        (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot))[None]
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _prepare_append(c, g, s):
    T, B, Hq, Hkv, D = c["T"], c["B"], c["Hq"], c["Hkv"], c["D"]
    if B == 1:                 # a prompt: T tokens after `past` ones
        pos = c["past"] + torch.arange(T, device=DEV)
        seq = torch.zeros(T, device=DEV, dtype=torch.int64)
    else:                      # decode: one token for each sequence
        pos = torch.randint(0, c["past"] + 1, (T,), generator=g, device=DEV)
        seq = torch.arange(T, device=DEV)
    cols = _pages(c["past"] + T if B == 1 else c["past"] + 1, c["page"])
    n_pages = B * cols + 1
    s["cache"] = _cache(c, g, n_pages)
    s["table"] = torch.randperm(n_pages, generator=g, device=DEV)[:B * cols].view(B, cols).int()
    s["pos"], s["seq"] = pos.int(), seq.int()
    # q, k and v as the fused projection leaves them: one row of (Hq + 2 Hkv) heads a token
    s["qkv"] = _normal(g, T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
    s["rope"] = _rope_table(c["past"] + T + 1, c["rot"])
    s["q_out"] = torch.empty((T, Hq, D), device=DEV, dtype=torch.bfloat16)


def _prepare_attn(c, g, s):
    B, Q, P, page = c["B"], c["Q"], c["prefix"], c["page"]
    last = torch.tensor(_last(c), device=DEV)
    n_keys = P + max(c["own_max"], c["Q"])
    cols, shared = _pages(n_keys, page), P // page      # whole pages are shared
    n_pages = _pages(P, page) + B * (cols - shared) + 1
    s["cache"] = _cache(c, g, n_pages)
    perm = torch.randperm(n_pages, generator=g, device=DEV).int()
    s["prefix"] = perm[:_pages(P, page)].contiguous()
    mine = perm[_pages(P, page):][:B * (cols - shared)].view(B, cols - shared)
    s["table"] = torch.cat([s["prefix"][:shared].expand(B, shared), mine], 1).contiguous()
    pos = last[:, None] - (Q - 1) + torch.arange(Q, device=DEV)[None]
    s["pos"] = torch.where(last[:, None] < 0, torch.full_like(pos, -1), pos).reshape(-1).int()
    s["q"] = (2.0 * _normal(g, B * Q, c["Hq"], c["D"])).to(torch.bfloat16)
    s["n_keys"], s["sm"] = n_keys, 1.0 / math.sqrt(c["D"])


def _prepare_logprobs(c, g, s):
    z = 2.5 * _normal(g, c["T"], c["V"])
    s["z"] = z.to(torch.bfloat16) if c["dtype"] == "bf16" else z
    s["tok"] = torch.randint(0, c["V"], (c["T"],), generator=g, device=DEV, dtype=torch.int32)


def _handles(c, s):
    """What a program keeps for the library's calls: descriptors, outputs and workspaces."""
    import bit_expert_ffn_moe_amd as moe
    s["moe"] = moe
    if c["op"] == "linear":
        fmt = moe.MOE_W_FP4_E2M1_UE8M0_K32 if c["fmt"] == "fp4" else moe.MOE_W_INT4_BF16_GROUP
        s["w"] = moe.make_w4(fmt, c["N"], c["K"], c["group"], s["q"], s["scale"], s["zero"])
        s["dt"] = moe.MOE_DT_BF16 if c["out"] == "bf16" else moe.MOE_DT_F32
        s["y"] = torch.empty((c["T"], c["N"]), device=DEV,
                             dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    elif c["op"] in ("append", "attn"):
        k = s["cache"]
        s["kv"] = moe.make_kv_cache(
            moe.MOE_DT_BF16 if c["cache"] == "bf16" else moe.MOE_DT_FP8_E4M3, k["k"].shape[0],
            c["page"], c["Hkv"], c["D"], k["k"], k["v"], k["ks"], k["vs"])
        if c["op"] == "append":
            s["style"] = moe.ROPE_HALF if c["style"] == "half" else moe.ROPE_PAIRS
        else:
            s["ws_bytes"] = moe.attn_workspace_bytes(s["kv"], c["B"], c["Q"], c["Hq"], c["prefix"],
                                                     s["n_keys"])
            s["ws"] = torch.empty(s["ws_bytes"], device=DEV, dtype=torch.uint8)
            s["o"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], device=DEV)
    else:
        s["dt"] = moe.MOE_DT_BF16 if c["dtype"] == "bf16" else moe.MOE_DT_F32
        s["ws_bytes"] = moe.token_logprobs_workspace_bytes(c["T"], c["V"], c["top"])
        s["ws"] = torch.empty(s["ws_bytes"], device=DEV, dtype=torch.uint8)
        s["lp"] = torch.empty(c["T"], device=DEV)
        s["ent"] = torch.empty(c["T"], device=DEV)
        s["ids"] = torch.empty((c["T"], c["top"]), device=DEV, dtype=torch.int32)
        s["tlp"] = torch.empty((c["T"], c["top"]), device=DEV)


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["c"]
    if own:
        return {"linear": _own_linear, "append": _own_append, "attn": _own_attn,
                "logprobs": _own_logprobs}[state["op"]](c, state)
    return {"linear": _plain_linear, "append": _plain_append, "attn": _plain_attn,
            "logprobs": _plain_logprobs}[state["op"]](c, state)


def _own_linear(c, s):
    s["moe"].w4_linear(s["w"], s["x"], c["K"], c["T"], s["y"], c["N"], s["dt"])
    return s["y"]


def _own_append(c, s):
    Hq, Hkv, D, qkv, k = c["Hq"], c["Hkv"], c["D"], s["qkv"], s["cache"]
    row = (Hq + 2 * Hkv) * D
    at = qkv.data_ptr()
    s["moe"].kv_append_rope(s["kv"], at, row, Hq, at + 2 * Hq * D, row, at + 2 * (Hq + Hkv) * D, row,
                            c["T"], s["rope"], s["rope"].shape[0], c["rot"], s["style"], s["seq"],
                            s["pos"], s["table"], s["table"].shape[0], s["table"].shape[1],
                            s["q_out"], None)
    return [s["q_out"], k["k"], k["v"], k["ks"], k["vs"]]


def _own_attn(c, s):
    s["moe"].attn_shared_prefix(s["kv"], s["q"], c["Hq"] * c["D"], c["B"], c["Q"], c["Hq"], s["pos"],
                                s["prefix"], c["prefix"], s["table"], s["table"].shape[1],
                                s["n_keys"], s["sm"], s["o"], s["lse"], None, s["ws"], s["ws_bytes"])
    return s["o"], s["lse"]


def _own_logprobs(c, s):
    s["moe"].token_logprobs(s["z"], s["dt"], c["V"], c["T"], c["V"], s["tok"], c["top"], s["lp"],
                            s["ent"], s["ids"], s["tlp"], None, s["ws"], s["ws_bytes"])
    return [s["lp"], s["ent"], s["ids"], s["tlp"]]


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _plain_linear(c, s):
    N, K, G, q = c["N"], c["K"], c["group"], s["q"]
    codes = torch.stack([q & 15, q >> 4], -1).view(N, K)
    at = torch.arange(K, device=DEV) // G
    if c["fmt"] == "fp4":
        w = torch.tensor(E2M1, device=DEV)[codes.int()]
        w = w * torch.exp2(s["scale"].float() - 127.0)[:, at]
    else:
        z = s["zero"].float()[:, at] if s["zero"] is not None else 8.0
        w = (codes.float() - z) * s["scale"].float()[:, at]
    y = s["x"].float() @ w.T
    return y.to(torch.bfloat16) if c["out"] == "bf16" else y


def _rotated(x, cos, sin, rot, style):
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if style == "half" else \
        (x[..., 0:rot:2], x[..., 1:rot:2])
    p, q = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([p, q], -1) if style == "half" else torch.stack([p, q], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_append(c, s):
    T, Hq, Hkv, D, k = c["T"], c["Hq"], c["Hkv"], c["D"], s["cache"]
    pos, seq = s["pos"].long(), s["seq"].long()
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    cs = s["rope"][pos][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:]
    qk = _rotated(x[:, :Hq + Hkv], cos, sin, c["rot"], c["style"])
    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    s["q_out"].copy_(qk[:, :Hq])
    kn, vn = qk[:, Hq:], x[:, Hq + Hkv:]
    if c["cache"] == "bf16":
        k["k"][page, :, slot] = kn.to(torch.bfloat16)
        k["v"][page, :, slot] = vn.to(torch.bfloat16)
        return [s["q_out"], k["k"], k["v"], None, None]
    ks, vs = kn.abs().amax(-1) / 448.0, vn.abs().amax(-1) / 448.0
    k["ks"][page, :, slot], k["vs"][page, :, slot] = ks, vs
    k["k"].view(torch.uint8)[page, :, slot] = (kn / ks[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    k["v"].view(torch.uint8)[page, :, slot] = (vn / vs[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return [s["q_out"], k["k"], k["v"], k["ks"], k["vs"]]


def _plain_attn(c, s):
    B, Q, Hq, Hkv, D, P, page = (c[n] for n in ("B", "Q", "Hq", "Hkv", "D", "prefix", "page"))
    G, n, k = Hq // Hkv, s["n_keys"], s["cache"]

    def values(a, scale, pages):        # pages [..., n] -> keys [..., Hkv, n * page, D] in fp32
        x = a[pages].float() if scale is None else a[pages].float() * scale[pages][..., None]
        return x.transpose(-4, -3).flatten(-3, -2)

    first = P // page                   # the first page of a sequence's own keys
    pre, mine = s["prefix"].long(), s["table"][:, first:].long()
    q = s["q"].float().view(B, Q, Hkv, G, D).permute(0, 2, 1, 3, 4)          # B Hkv Q G D
    qp = q.transpose(0, 1).reshape(Hkv, B * Q * G, D)
    kp, vp = (values(k[a], k[b], pre)[:, :P] for a, b in (("k", "ks"), ("v", "vs")))
    km, vm = (values(k[a], k[b], mine)[:, :, P - first * page:n - first * page]
              for a, b in (("k", "ks"), ("v", "vs")))
    sp = (qp @ kp.transpose(1, 2)).view(Hkv, B, Q, G, P).transpose(0, 1)
    so = (q.reshape(B, Hkv, Q * G, D) @ km.transpose(2, 3)).view(B, Hkv, Q, G, n - P)
    sc = torch.cat([sp, so], -1) * s["sm"]
    seen = torch.arange(n, device=DEV) <= s["pos"].view(B, 1, Q, 1, 1)
    sc = sc.masked_fill(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - m.clamp_min(-3e38))
    total = e.sum(-1, keepdim=True)
    pr = torch.where(total > 0, e / total, 0.0)
    op = pr[..., :P].transpose(0, 1).reshape(Hkv, B * Q * G, P) @ vp
    oo = pr[..., P:].reshape(B, Hkv, Q * G, n - P) @ vm
    o = op.view(Hkv, B, Q, G, D).transpose(0, 1) + oo.view(B, Hkv, Q, G, D)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * Q, Hq, D).to(torch.bfloat16)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(B * Q, Hq)
    return o, lse


def _plain_logprobs(c, s):
    z = s["z"].float()
    d = z - z.amax(1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lt = torch.log(total)
    lp = (d.gather(1, s["tok"].long()[:, None]) - lt)[:, 0]
    entropy = lt[:, 0] - (e * d).sum(1) / total[:, 0]
    # ties to the lowest id: one whole-number key of the value's order and the id turned round
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    key = order * (1 << 32) + ((1 << 32) - 1 - torch.arange(c["V"], device=DEV))
    ids = ((1 << 32) - 1 - torch.topk(key, c["top"], dim=1).values % (1 << 32))
    return [lp, entropy, ids.int(), d.gather(1, ids) - lt]


# ---------------------------------------------------------------- work and exact values

def work(c):
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        n_g = -(-K // c["group"])
        per = 1 if c["fmt"] == "fp4" else 3 if c["zeros"] else 2
        return {"bytes": N * K // 2 + N * n_g * per + T * K * 2 + T * N * (2 if c["out"] == "bf16" else 4),
                "flops": 2 * T * N * K}
    if c["op"] == "append":
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        row = 2 * D if c["cache"] == "bf16" else D + 4
        return {"bytes": T * (2 * Hq * 2 * D + 2 * Hkv * (2 * D + row) + c["rot"] * 4 + 12),
                "flops": T * (Hq + Hkv) * c["rot"] * 3}
    if c["op"] == "attn":
        B, Q, Hq, Hkv, D, P = (c[n] for n in ("B", "Q", "Hq", "Hkv", "D", "prefix"))
        last = [p for p in _last(c) if p >= 0]
        row = 2 * Hkv * (2 * D if c["cache"] == "bf16" else D + 4)
        keys = P + sum(p + 1 - P for p in last)
        seen = sum((p + 1) * Q - Q * (Q - 1) // 2 for p in last)
        return {"bytes": keys * row + B * Q * Hq * (4 * D + 4), "flops": 4 * D * Hq * seen}
    T, V = c["T"], c["V"]
    return {"bytes": T * V * (2 if c["dtype"] == "bf16" else 4) + T * (12 + 8 * c["top"]),
            "flops": 6 * T * V}


def exact(case, seed):
    """What run() returns, from the operators' definitions in 64 bits."""
    s = {"c": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    {"linear": _prepare_linear, "append": _prepare_append, "attn": _prepare_attn,
     "logprobs": _prepare_logprobs}[case["op"]](case, g, s)
    return {"linear": _exact_linear, "append": _exact_append, "attn": _exact_attn,
            "logprobs": _exact_logprobs}[case["op"]](case, s)


def _exact_linear(c, s):
    """Group by group: x's part times the group's codes, then the group's scale."""
    N, K, G = c["N"], c["K"], c["group"]
    y = torch.zeros((c["T"], N), device=DEV, dtype=torch.float64)
    for j in range(-(-K // G)):
        lo, hi = j * G, min(K, (j + 1) * G)
        b = s["q"][:, lo // 2:hi // 2].int()
        w = torch.empty((N, hi - lo), device=DEV, dtype=torch.float64)
        for half in (0, 1):
            n = (b >> (4 * half)) & 15
            if c["fmt"] == "fp4":       # sign, two bits of exponent, one of mantissa
                e, m = ((n >> 1) & 3).double(), (n & 1).double()
                mag = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)
                w[:, half::2] = torch.where(n >= 8, -mag, mag)
            else:
                w[:, half::2] = n.double() - (s["zero"][:, j, None].double() if c["zeros"] else 8.0)
        scale = 2.0 ** (s["scale"][:, j].double() - 127) if c["fmt"] == "fp4" else s["scale"][:, j].double()
        y += (s["x"][:, lo:hi].double() @ w.T) * scale
    return y


def _exact_append(c, s):
    T, Hq, Hkv, D, R = c["T"], c["Hq"], c["Hkv"], c["D"], c["rot"]
    x = s["qkv"].double().view(T, -1, D)
    out = x.clone()
    t = s["rope"].double()[s["pos"].long()]
    for i in range(R // 2):             # pair by pair, a rotation of the plane
        i0, i1 = (i, i + R // 2) if c["style"] == "half" else (2 * i, 2 * i + 1)
        turn = torch.complex(t[:, i], t[:, R // 2 + i])[:, None]
        z = torch.complex(x[:, :Hq + Hkv, i0], x[:, :Hq + Hkv, i1]) * turn
        out[:, :Hq + Hkv, i0], out[:, :Hq + Hkv, i1] = z.real, z.imag
    page = s["table"].long()[s["seq"].long(), (s["pos"] // c["page"]).long()]
    slot = (s["pos"] % c["page"]).long()
    got = [out[:, :Hq]]
    scales = []
    for a, sc, lo in (("k", "ks", Hq), ("v", "vs", Hq + Hkv)):
        new, buf = out[:, lo:lo + Hkv], s["cache"][a].double()
        if c["cache"] == "fp8":
            amax = new.abs().max(-1).values
            new = new * (448.0 / amax)[..., None]
            sb = s["cache"][sc].double()
            sb[page, :, slot] = amax / 448.0
            scales.append(sb)
        buf[page, :, slot] = new
        got.append(buf)
    return got + (scales or [None, None])


def _exact_attn(c, s):
    """Sequence by sequence and head by head, the keys in one row."""
    B, Q, Hq, Hkv, D, P, page = (c[n] for n in ("B", "Q", "Hq", "Hkv", "D", "prefix", "page"))
    if B * Hq * (P + c["own_max"]) * Q > 3e8:
        return None
    o = torch.zeros((B * Q, Hq, D), device=DEV, dtype=torch.float64)
    lse = torch.full((B * Q, Hq), -math.inf, device=DEV, dtype=torch.float64)
    k, pos = s["cache"], s["pos"].tolist()
    for b in range(B):
        n = max(pos[b * Q:(b + 1) * Q]) + 1
        if n <= 0:
            continue
        j = torch.arange(n, device=DEV)
        pg = torch.where(j < P, s["prefix"][(j // page).clamp_max(len(s["prefix"]) - 1)],
                         s["table"][b][j // page]).long()
        for h in range(Hkv):
            kk, vv = k["k"][pg, h, j % page].double(), k["v"][pg, h, j % page].double()
            if c["cache"] == "fp8":
                kk *= k["ks"][pg, h, j % page].double()[:, None]
                vv *= k["vs"][pg, h, j % page].double()[:, None]
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            for i in range(Q):
                t = b * Q + i
                a = s["q"][t, hs].double() @ kk[:pos[t] + 1].T * s["sm"]
                o[t, hs] = torch.softmax(a, 1) @ vv[:pos[t] + 1]
                lse[t, hs] = torch.logsumexp(a, 1)
    return o, lse


def _exact_logprobs(c, s):
    got = [[], [], [], []]
    for lo in range(0, c["T"], 512):
        z = s["z"][lo:lo + 512].double()
        lp = torch.log_softmax(z, 1)
        got[0].append(lp.gather(1, s["tok"][lo:lo + 512].long()[:, None])[:, 0])
        got[1].append(-(lp.exp() * lp).sum(1))
        got[3].append(torch.sort(lp, 1, descending=True).values[:, :c["top"]])
    return [torch.cat(got[0]), torch.cat(got[1]), None, torch.cat(got[3])]
