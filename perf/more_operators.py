"""What is measured of the operators that stand between the decode step's projections, cache and
log probabilities: the residual's addition with the root-mean-square norm, low-rank adapters of
many requests beside a shared projection, attention over a cache held in 4 bits, and the penalties,
biases and grammar masks on logits.

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
        # one decode token of the layer's hidden width, ready for the experts: latency
        dict(name="norm_t1", op="norm", T=1, H=4096, res="bf16", y=True, q=True),
        # a ragged batch of a width that is no multiple of 128, residual stream in fp32
        dict(name="norm_t37_odd", op="norm", T=37, H=2088, res="f32", y=True, q=False),
        # a prompt of 8192 tokens between attention and experts: the largest
        dict(name="norm_prompt_t8192", op="norm", T=8192, H=4096, res="bf16", y=True, q=True),
        # one token of one request with an adapter of rank 16: latency
        dict(name="lora_t1_r16", op="lora", T=1, K=4096, N=4096, adapters=8, max_rank=16, mixed=False,
             runs=False, out="bf16"),
        # fused q/k/v projection of 32 decoding requests, 24 adapters of ranks up to 64 among them,
        # some requests without one
        dict(name="lora_decode_t32", op="lora", T=32, K=4096, N=6144, adapters=24, max_rank=64,
             mixed=True, runs=False, out="bf16"),
        # prompts of several requests in one batch, each with its adapter
        dict(name="lora_prompt_t4096", op="lora", T=4096, K=4096, N=4096, adapters=6, max_rank=32,
             mixed=False, runs=True, out="bf16"),
        # one request's next token: a short history, no grammar: latency
        dict(name="logits_t1", op="logits", dtype="f32", T=1, V=131072, history=600, bias=0, mask=False),
        # a batch with an odd vocabulary, penalties, biases and a grammar mask for half of the rows
        dict(name="logits_t32_odd", op="logits", dtype="bf16", T=32, V=50021, history=2000, bias=20,
             mask=True),
        # verification of a large batch: long histories, everything on
        dict(name="logits_t256", op="logits", dtype="f32", T=256, V=131072, history=4096, bias=100,
             mask=True),
        # a small batch behind a short system prompt that ends inside a page: latency
        dict(name="attn4_small_b4", op="attn", B=4, Q=1, Hq=8, Hkv=2, D=64, page=16, prefix=500,
             own_max=60, pad=True),
        # ordinary decode: 32 sequences of up to 2048 tokens of their own behind 8192 shared ones
        dict(name="attn4_decode_b32", op="attn", B=32, Q=1, Hq=32, Hkv=8, D=128, page=64,
             prefix=8192, own_max=2048, pad=False),
        # why a cache is held in 4 bits: 8 sequences of up to 65536 tokens, nothing shared
        dict(name="attn4_long_b8", op="attn", B=8, Q=1, Hq=64, Hkv=8, D=128, page=64, prefix=0,
             own_max=65536, pad=False),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    op = rng.choice(["norm", "lora", "lora", "logits", "attn", "attn"])
    if op == "norm":
        H = rng.choice([8 * _logu(rng, 16, 1024), 128 * _logu(rng, 1, 64)])
        q = H % 128 == 0 and rng.random() < 0.7
        return dict(op=op, T=_logu(rng, 1, max(1, min(8192, 8192 * 4096 // H))), H=H,
                    res=rng.choice(["bf16", "f32"]) if H * 4 <= 16384 else "bf16",
                    y=not q or rng.random() < 0.7, q=q)
    if op == "lora":
        T = _logu(rng, 1, 4096)
        return dict(op=op, T=T, K=8 * _logu(rng, 16, 512), N=_logu(rng, 64, 4096),
                    adapters=_logu(rng, 1, 32), max_rank=rng.choice([8, 16, 32, 64] if T < 2048 else [8, 16, 32]),
                    mixed=rng.random() < 0.5, runs=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
    if op == "logits":
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), T=_logu(rng, 1, 256),
                    V=_logu(rng, 1000, 131072), history=_logu(rng, 1, 4096),
                    bias=rng.choice([0, 1, 20, 100]), mask=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8])
    return dict(op=op, B=_logu(rng, 1, 32), Q=rng.choice([1, 1, 2, 4]), Hq=Hkv * G, Hkv=Hkv,
                D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                prefix=_logu(rng, 16, 16384), own_max=_logu(rng, 8, 4096), pad=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"c": case, "op": case["op"]}
    {"norm": _prepare_norm, "lora": _prepare_lora, "attn": _prepare_attn,
     "logits": _prepare_logits}[case["op"]](case, g, s)
    if own:
        _handles(case, s)
    return s


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _prepare_norm(c, g, s):
    T, H = c["T"], c["H"]
    s["x"] = _normal(g, T, H).to(torch.bfloat16)
    # a residual stream of several layers, larger than one block's output
    s["res"] = (4.0 * _normal(g, T, H)).to(torch.bfloat16 if c["res"] == "bf16" else torch.float32)
    s["w"] = (1.0 + 0.2 * _normal(g, H)).to(torch.bfloat16)
    s["eps"] = 1e-6


def _prepare_lora(c, g, s):
    T, K, N, n, R = c["T"], c["K"], c["N"], c["adapters"], c["max_rank"]
    s["x"] = _normal(g, T, K).to(torch.bfloat16)
    s["base"] = _normal(g, T, N).to(torch.bfloat16 if c["out"] == "bf16" else torch.float32)
    s["a"] = (_normal(g, n, R, K) / math.sqrt(K)).to(torch.bfloat16)
    s["b"] = (0.1 * _normal(g, n, N, R)).to(torch.bfloat16)
    s["rank"] = torch.minimum(_ints(g, 1, 9, n) * ((R + 7) // 8), torch.full((n,), R, device=DEV)).int() \
        if c["mixed"] else None
    s["scale"] = 0.5 + torch.rand(n, generator=g, device=DEV)
    if c["runs"]:                       # prompts behind each other: runs of tokens of one adapter
        cut = torch.sort(torch.randint(0, T + 1, (min(n, T),), generator=g, device=DEV)).values
        s["of"] = (torch.searchsorted(cut, torch.arange(T, device=DEV), right=True) % n).int()
    else:                               # a request in eight has none
        of = _ints(g, 0, n, T)
        s["of"] = torch.where(torch.rand(T, generator=g, device=DEV) < 0.125, torch.full_like(of, -1), of) \
            if T > 1 else of


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


def _fp4_rows(x):
    """Rows as an append leaves them in a 4-bit cache: per 32 columns the smallest power of two that
    brings the largest to 6 at most, E2M1 codes to nearest even, two a byte."""
    g = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(g.abs().amax(-1))
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 125)
    u = torch.ldexp(g.abs(), -e[..., None].float())
    code = (u > 0.25).to(torch.uint8)
    code += u >= 0.75
    code += u > 1.25
    code += u >= 1.75
    code += u > 2.5
    code += u >= 3.5
    code += u > 5.0
    code += 8 * (g < 0)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8)


def _prepare_attn(c, g, s):
    B, Q, P, page = c["B"], c["Q"], c["prefix"], c["page"]
    last = torch.tensor(_last(c), device=DEV)
    n_keys = P + max(c["own_max"], c["Q"])
    cols, shared = _pages(n_keys, page), P // page      # whole pages are shared
    n_pages = _pages(P, page) + B * (cols - shared) + 1
    shape = (n_pages, c["Hkv"], page, c["D"])
    (k, ks), (v, vs) = _fp4_rows(_normal(g, *shape)), _fp4_rows(_normal(g, *shape))
    s["cache"] = dict(k=k, ks=ks, v=v, vs=vs)
    perm = torch.randperm(n_pages, generator=g, device=DEV).int()
    s["prefix"] = perm[:_pages(P, page)].contiguous()
    mine = perm[_pages(P, page):][:B * (cols - shared)].view(B, cols - shared)
    s["table"] = torch.cat([s["prefix"][:shared].expand(B, shared), mine], 1).contiguous()
    pos = last[:, None] - (Q - 1) + torch.arange(Q, device=DEV)[None]
    s["pos"] = torch.where(last[:, None] < 0, torch.full_like(pos, -1), pos).reshape(-1).int()
    s["q"] = (2.0 * _normal(g, B * Q, c["Hq"], c["D"])).to(torch.bfloat16)
    s["n_keys"], s["sm"] = n_keys, 1.0 / math.sqrt(c["D"])


def _prepare_logits(c, g, s):
    T, V, n = c["T"], c["V"], c["history"]
    z = 2.5 * _normal(g, T, V)
    s["z"] = z.to(torch.bfloat16) if c["dtype"] == "bf16" else z
    # texts repeat themselves: ids spread over their logarithm, half a history to a whole one long
    u = torch.rand((T, n), generator=g, device=DEV)
    s["history"] = ((V ** u).int() - 1).clamp(0, V - 1)
    s["n_tokens"] = _ints(g, max(1, n // 2), n + 1, T)
    s["n_prompt"] = (s["n_tokens"] * torch.rand(T, generator=g, device=DEV)).int()
    s["seq"] = torch.randperm(T, generator=g, device=DEV).int()
    s["repetition"] = 1.0 + 0.3 * torch.rand(T, generator=g, device=DEV)
    s["presence"] = 0.5 * torch.rand(T, generator=g, device=DEV)
    s["frequency"] = 0.3 * torch.rand(T, generator=g, device=DEV)
    if c["bias"]:                       # different ids within a row
        first = _ints(g, 0, V, T, 1).long()
        s["bias_ids"] = ((first + torch.arange(c["bias"], device=DEV) * (V // c["bias"])) % V).int()
        s["bias"] = 3.0 * _normal(g, T, c["bias"])
    if c["mask"]:                       # a grammar's state allows an eighth of the ids, or has no mask
        n_m = max(1, T // 2)
        w = [_ints(g, -(1 << 31), (1 << 31) - 1, n_m, -(-V // 32)) for _ in range(3)]
        s["mask"] = w[0] & w[1] & w[2]
        s["mask_of"] = torch.where(_ints(g, 0, 2, T) > 0, _ints(g, 0, n_m, T),
                                   torch.full((T,), -1, device=DEV, dtype=torch.int32))


def _handles(c, s):
    """What a program keeps for the library's calls: descriptors, outputs and workspaces."""
    import bit_expert_ffn_moe_amd as moe
    s["moe"] = moe
    dt = {"bf16": moe.MOE_DT_BF16, "f32": moe.MOE_DT_F32}
    if c["op"] == "norm":
        s["dt"] = dt[c["res"]]
        s["res_out"] = torch.empty_like(s["res"])
        s["y"] = torch.empty_like(s["x"]) if c["y"] else None
        s["q"] = torch.empty(s["x"].shape, device=DEV, dtype=torch.float8_e4m3fn) if c["q"] else None
        s["qs"] = torch.empty((c["T"], c["H"] // 128), device=DEV) if c["q"] else None
    elif c["op"] == "lora":
        s["dt"] = dt[c["out"]]
        s["w"] = moe.make_lora(c["adapters"], c["max_rank"], c["K"], c["N"], s["a"], s["b"], s["rank"],
                               s["scale"])
        s["y"] = torch.empty_like(s["base"])
        s["ws_bytes"] = moe.lora_workspace_bytes(s["w"], c["T"])
        s["ws"] = torch.empty(s["ws_bytes"], device=DEV, dtype=torch.uint8)
    elif c["op"] == "attn":
        k = s["cache"]
        s["kv"] = moe.make_kv_cache(moe.MOE_DT_FP4_E2M1, k["k"].shape[0], c["page"], c["Hkv"], c["D"],
                                    k["k"], k["v"], k["ks"], k["vs"])
        s["ws_bytes"] = moe.attn_workspace_bytes(s["kv"], c["B"], c["Q"], c["Hq"], c["prefix"],
                                                 s["n_keys"])
        s["ws"] = torch.empty(s["ws_bytes"], device=DEV, dtype=torch.uint8)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device=DEV)
    else:
        s["dt"] = dt[c["dtype"]]
        more = dict(bias_ids=s["bias_ids"], bias=s["bias"], n_bias=c["bias"]) if c["bias"] else {}
        if c["mask"]:
            more.update(mask=s["mask"], mask_stride=s["mask"].shape[1], n_masks=s["mask"].shape[0],
                        mask_of=s["mask_of"])
        s["rules"] = moe.make_logits_rules(
            history=s["history"], history_stride=c["history"], max_history=c["history"], n_seqs=c["T"],
            seq_of=s["seq"], n_tokens=s["n_tokens"], n_prompt=s["n_prompt"],
            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], **more)
        s["out"] = torch.empty_like(s["z"])


# ---------------------------------------------------------------- one pass

def run(state):
    c = state["c"]
    if own:
        return {"norm": _own_norm, "lora": _own_lora, "attn": _own_attn,
                "logits": _own_logits}[state["op"]](c, state)
    return {"norm": _plain_norm, "lora": _plain_lora, "attn": _plain_attn,
            "logits": _plain_logits}[state["op"]](c, state)


def _own_norm(c, s):
    s["moe"].add_rmsnorm(s["x"], c["H"], s["res"], s["dt"], c["H"], c["T"], c["H"], s["w"], s["eps"],
                         s["res_out"], s["y"], s["q"], s["qs"])
    return [s["res_out"], s["y"], s["q"], s["qs"]]


def _own_lora(c, s):
    s["moe"].lora_linear(s["w"], s["x"], c["K"], c["T"], s["of"], s["base"], c["N"], s["y"], c["N"],
                         s["dt"], None, s["ws"], s["ws_bytes"])
    return s["y"]


def _own_attn(c, s):
    s["moe"].attn_shared_prefix(s["kv"], s["q"], c["Hq"] * c["D"], c["B"], c["Q"], c["Hq"], s["pos"],
                                s["prefix"] if c["prefix"] else None, c["prefix"], s["table"],
                                s["table"].shape[1], s["n_keys"], s["sm"], s["o"], s["lse"], None,
                                s["ws"], s["ws_bytes"])
    return s["o"], s["lse"]


def _own_logits(c, s):
    s["moe"].logits_adjust(s["rules"], s["z"], s["dt"], c["V"], c["T"], c["V"], s["out"], s["dt"],
                           c["V"], None)
    return s["out"]


def _plain_norm(c, s):
    """The residual stream is stored in its type, and the norm is of what is stored."""
    r = (s["x"].float() + s["res"].float()).to(s["res"].dtype)
    x = r.float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"]) * s["w"].float()
    q = sc = None
    if c["q"]:
        b = y.view(c["T"], -1, 128)
        sc = b.abs().amax(2) / 448.0
        q = (b / sc[..., None]).to(torch.float8_e4m3fn).view(c["T"], -1)
    return [r, y.to(torch.bfloat16) if c["y"] else None, q, sc]


def _plain_lora(c, s):
    """All adapters at once; what is not of a token's adapter, or past its rank, is put out between
    the two products."""
    n, R = c["adapters"], c["max_rank"]
    h = s["x"].float() @ s["a"].view(n * R, -1).float().T
    keep = s["of"].view(-1, 1, 1) == torch.arange(n, device=DEV).view(1, n, 1)
    if s["rank"] is not None:
        keep = keep & (torch.arange(R, device=DEV) < s["rank"].view(n, 1))
    h = torch.where(keep, h.view(-1, n, R) * s["scale"].view(n, 1), 0.0).view(-1, n * R)
    y = s["base"].float() + h @ s["b"].float().transpose(1, 2).reshape(n * R, -1)
    return y.to(s["base"].dtype)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _plain_attn(c, s):
    B, Q, Hq, Hkv, D, P, page = (c[n] for n in ("B", "Q", "Hq", "Hkv", "D", "prefix", "page"))
    G, n, k = Hq // Hkv, s["n_keys"], s["cache"]
    two = torch.tensor([(a, b) for b in E2M1 for a in E2M1], device=DEV)     # the values of a byte

    def values(a, scale, pages):        # pages [..., n] -> keys [..., Hkv, n * page, D] in fp32
        x = two[a[pages].int()].flatten(-2).unflatten(-1, (-1, 32))
        x = (x * torch.exp2(scale[pages].float() - 127.0)[..., None]).flatten(-2)
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


def _plain_logits(c, s):
    T, V = c["T"], c["V"]
    at = torch.arange(c["history"], device=DEV)
    ids = s["history"][s["seq"].long()].long()
    inside = at < s["n_tokens"][:, None]
    made = (inside & (at >= s["n_prompt"][:, None])).float()
    count = torch.zeros((T, V), device=DEV).scatter_add_(1, ids, made)
    seen = torch.zeros((T, V), device=DEV).scatter_add_(1, ids, inside.float()) > 0
    z = s["z"].float()
    if c["bias"]:
        z = z.scatter_add(1, s["bias_ids"].long(), s["bias"])
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - (s["presence"][:, None] * (count > 0) + s["frequency"][:, None] * count)
    if c["mask"]:
        bits = (s["mask"][s["mask_of"].clamp_min(0).long()][:, :, None]
                >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        out = (bits.view(T, -1)[:, :V] == 0) & (s["mask_of"] >= 0)[:, None]
        z = z.masked_fill(out, -math.inf)
    return z.to(s["z"].dtype)


# ---------------------------------------------------------------- work and exact values

def work(c):
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        out = (2 if c["y"] else 0) + (1 + 4 / 128 if c["q"] else 0)
        return {"bytes": T * H * (2 + 2 * (2 if c["res"] == "bf16" else 4) + out) + 2 * H,
                "flops": T * H * 5}
    if c["op"] == "lora":
        T, K, N, R = c["T"], c["K"], c["N"], c["max_rank"]
        used = min(c["adapters"], T)
        per = R * (9 / 16 if c["mixed"] else 1)      # ranks of a mixed set: an eighth to the whole
        return {"bytes": T * K * 2 + T * N * 2 * (2 if c["out"] == "bf16" else 4)
                + int(used * per) * (K + N) * 2, "flops": int(2 * T * per * (K + N))}
    if c["op"] == "attn":
        B, Q, Hq, Hkv, D, P = (c[n] for n in ("B", "Q", "Hq", "Hkv", "D", "prefix"))
        last = [p for p in _last(c) if p >= 0]
        row = 2 * Hkv * (D // 2 + D // 32)
        keys = P + sum(p + 1 - P for p in last)
        seen = sum((p + 1) * Q - Q * (Q - 1) // 2 for p in last)
        return {"bytes": keys * row + B * Q * Hq * (4 * D + 4), "flops": 4 * D * Hq * seen}
    T, V = c["T"], c["V"]
    return {"bytes": T * V * 2 * (2 if c["dtype"] == "bf16" else 4) + T * 3 * c["history"]
            + T * 8 * c["bias"] + (max(1, T // 2) * -(-V // 32) * 4 if c["mask"] else 0),
            "flops": 6 * T * V}


def exact(case, seed):
    """What run() returns, from the operators' definitions in 64 bits."""
    s = {"c": case}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    {"norm": _prepare_norm, "lora": _prepare_lora, "attn": _prepare_attn,
     "logits": _prepare_logits}[case["op"]](case, g, s)
    return {"norm": _exact_norm, "lora": _exact_lora, "attn": _exact_attn,
            "logits": _exact_logits}[case["op"]](case, s)


def _exact_norm(c, s):
    total = s["x"].double() + s["res"].double()
    stored = total.to(s["res"].dtype).double()      # what the norm is of
    y = torch.empty_like(stored)
    for lo in range(0, c["T"], 1024):
        r = stored[lo:lo + 1024]
        y[lo:lo + 1024] = r / torch.sqrt((r * r).sum(1, keepdim=True) / c["H"] + s["eps"]) * s["w"].double()
    q = sc = None
    if c["q"]:
        top = y.abs().unflatten(1, (-1, 128)).max(2).values
        sc, q = top / 448.0, (y.unflatten(1, (-1, 128)) * (448.0 / top)[..., None]).flatten(1)
    return [total, y if c["y"] else None, q, sc]


def _exact_lora(c, s):
    y = s["base"].double()
    for i in range(c["adapters"]):
        t = torch.nonzero(s["of"] == i)[:, 0]
        r = int(s["rank"][i]) if s["rank"] is not None else c["max_rank"]
        h = s["x"][t].double() @ s["a"][i, :r].double().T
        y[t] += (h @ s["b"][i, :, :r].double().T) * s["scale"][i].double()
    return y


def _exact_attn(c, s):
    """Sequence by sequence and head by head, the keys in one row."""
    B, Q, Hq, Hkv, D, P, page = (c[n] for n in ("B", "Q", "Hq", "Hkv", "D", "prefix", "page"))
    if B * Hq * (P + c["own_max"]) * Q > 3e8:
        return None
    o = torch.zeros((B * Q, Hq, D), device=DEV, dtype=torch.float64)
    lse = torch.full((B * Q, Hq), -math.inf, device=DEV, dtype=torch.float64)
    pos = s["pos"].tolist()

    def rows(a, scale, pg, h, slot):    # sign, two bits of exponent, one of mantissa
        b = s["cache"][a][pg, h, slot].int()
        n = torch.stack([b & 15, b >> 4], -1).flatten(-2)
        e, m = ((n >> 1) & 3).double(), (n & 1).double()
        x = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)
        x = torch.where(n >= 8, -x, x)
        return x * (2.0 ** (s["cache"][scale][pg, h, slot].double() - 127)).repeat_interleave(32, -1)

    for b in range(B):
        n = max(pos[b * Q:(b + 1) * Q]) + 1
        if n <= 0:
            continue
        j = torch.arange(n, device=DEV)
        pg = s["table"][b][j // page].long()
        if P:
            pg = torch.where(j < P, s["prefix"][(j // page).clamp_max(len(s["prefix"]) - 1)].long(), pg)
        for h in range(Hkv):
            kk, vv = rows("k", "ks", pg, h, j % page), rows("v", "vs", pg, h, j % page)
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            for i in range(Q):
                t = b * Q + i
                a = s["q"][t, hs].double() @ kk[:pos[t] + 1].T * s["sm"]
                o[t, hs] = torch.softmax(a, 1) @ vv[:pos[t] + 1]
                lse[t, hs] = torch.logsumexp(a, 1)
    return o, lse


def _exact_logits(c, s):
    """Row by row."""
    T, V = c["T"], c["V"]
    got = torch.empty((T, V), device=DEV, dtype=torch.float64)
    seq, total, prompt = s["seq"].tolist(), s["n_tokens"].tolist(), s["n_prompt"].tolist()
    state = s["mask_of"].tolist() if c["mask"] else [-1] * T
    for t in range(T):
        z = s["z"][t].double()
        if c["bias"]:
            z[s["bias_ids"][t].long()] += s["bias"][t].double()
        text = s["history"][seq[t], :total[t]].long()
        met = torch.unique(text)
        rep = s["repetition"][t].double()
        z[met] = torch.where(z[met] > 0, z[met] / rep, z[met] * rep)
        made = torch.bincount(text[prompt[t]:], minlength=V)
        z = torch.where(made > 0, z - s["presence"][t].double() - s["frequency"][t].double() * made, z)
        if state[t] >= 0:
            v = torch.arange(V, device=DEV)
            z[(s["mask"][state[t]].long()[v // 32] >> (v % 32)) & 1 == 0] = -math.inf
        got[t] = z
    return got
