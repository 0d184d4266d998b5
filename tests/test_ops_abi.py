"""CPU tests of the decode-step operators' argument checks: every refusal
happens on the host before any HIP call (no GPU needed), and empty batches
are accepted without a device."""
import ctypes

import pytest

moe = pytest.importorskip("bit_expert_ffn_moe_amd")

P, BIG = 0x100000, 1 << 40
EINVAL, ENOTSUP, EALIGN, EWS, OK = (moe.MOE_EINVAL, moe.MOE_ENOTSUP, moe.MOE_EALIGN,
                                    moe.MOE_EWORKSPACE, moe.MOE_OK)


def w4(**o):
    a = dict(fmt=1, N=64, K=128, group=32, q=P, scale=P, zero=None)
    a.update(o)
    return ctypes.byref(moe.make_w4(a["fmt"], a["N"], a["K"], a["group"], a["q"], a["scale"],
                                    a["zero"]))


@pytest.mark.parametrize("weights,call,expect", [
    ({}, dict(T=0), OK),
    (dict(fmt=2), {}, ENOTSUP),
    (dict(q=None), {}, EINVAL),
    (dict(scale=None), {}, EINVAL),
    (dict(K=48), {}, EINVAL),
    (dict(K=0), {}, EINVAL),
    (dict(N=0), {}, EINVAL),
    (dict(group=64), {}, EINVAL),
    (dict(zero=P), {}, EINVAL),
    (dict(fmt=3, group=48), {}, EINVAL),
    (dict(fmt=3, group=256), {}, EINVAL),
    (dict(fmt=3, group=64, zero=P), dict(T=0), OK),
    (dict(N=(1 << 20) + 1), dict(ys=1 << 21), ENOTSUP),
    (dict(K=(1 << 20) + 32), dict(xs=1 << 21), ENOTSUP),
    (dict(q=P + 8), {}, EALIGN),
    (dict(fmt=3, zero=P + 1), {}, EALIGN),
    ({}, dict(x=None), EINVAL),
    ({}, dict(y=None), EINVAL),
    ({}, dict(x=P + 2), EALIGN),
    ({}, dict(xs=127), EINVAL),
    ({}, dict(xs=132), EINVAL),
    ({}, dict(ys=63), EINVAL),
    ({}, dict(T=-1), EINVAL),
    ({}, dict(T=(1 << 18) + 1), ENOTSUP),
    ({}, dict(dt=3), EINVAL),
])
def test_w4_linear(weights, call, expect):
    c = dict(x=P, xs=128, T=4, y=P, ys=64, dt=2)
    c.update(call)
    assert moe.raw_call("w4_linear", w4(**weights), c["x"], c["xs"], c["T"], c["y"], c["ys"],
                        c["dt"], None) == expect


def test_w4_linear_null_descriptor():
    assert moe.raw_call("w4_linear", None, P, 128, 1, P, 64, 2, None) == EINVAL


def cache(**o):
    a = dict(dt=1, n=10, page=16, Hkv=2, D=64, k=P, v=P, ks=None, vs=None)
    a.update(o)
    return ctypes.byref(moe.make_kv_cache(a["dt"], a["n"], a["page"], a["Hkv"], a["D"], a["k"],
                                          a["v"], a["ks"], a["vs"]))


BAD_CACHES = [
    (dict(dt=2), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(n=0), EINVAL),
    (dict(page=24), EINVAL), (dict(page=8), ENOTSUP), (dict(page=2048), ENOTSUP),
    (dict(D=96), ENOTSUP), (dict(Hkv=0), EINVAL), (dict(Hkv=1025), ENOTSUP),
    (dict(ks=P), EINVAL), (dict(dt=3), EINVAL), (dict(dt=3, ks=P), EINVAL),
    (dict(dt=3, ks=P, vs=P + 4), EALIGN), (dict(k=P + 8), EALIGN),
]


def append(c, **o):
    a = dict(q=P, qs=256, Hq=4, k=P, ks=128, v=P, vs=128, T=3, rope=P, rows=9, R=64, style=1, seq=P,
             pos=P, table=P, B=2, cols=4, qo=P, st=None)
    a.update(o)
    return moe.raw_call("kv_append_rope", c, a["q"], a["qs"], a["Hq"], a["k"], a["ks"], a["v"],
                        a["vs"], a["T"], a["rope"], a["rows"], a["R"], a["style"], a["seq"],
                        a["pos"], a["table"], a["B"], a["cols"], a["qo"], a["st"], None)


@pytest.mark.parametrize("c,expect", BAD_CACHES)
def test_bad_caches(c, expect):
    assert append(cache(**c)) == expect
    assert attn(cache(**c)) == expect
    assert moe._lib.attn_workspace_bytes(cache(**c), 2, 1, 4, 20, 64) == 0


@pytest.mark.parametrize("o,expect", [
    (dict(T=0), OK), (dict(T=0, Hq=0, q=None, qo=None), OK),
    (dict(T=0, R=0, rope=None, rows=0, style=0), OK),
    (dict(T=-1), EINVAL), (dict(T=(1 << 18) + 1), ENOTSUP), (dict(k=None), EINVAL),
    (dict(v=None), EINVAL), (dict(seq=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(table=None), EINVAL), (dict(q=None), EINVAL), (dict(qo=None), EINVAL),
    (dict(Hq=0), EINVAL), (dict(Hq=1025, qs=1 << 20), ENOTSUP), (dict(R=24), EINVAL),
    (dict(R=80), EINVAL), (dict(R=-16), EINVAL), (dict(rope=None), EINVAL), (dict(rows=0), EINVAL),
    (dict(style=3), EINVAL), (dict(R=0), EINVAL), (dict(qs=248), EINVAL), (dict(qs=260), EINVAL),
    (dict(ks=120), EINVAL), (dict(vs=129), EINVAL), (dict(B=0), EINVAL), (dict(cols=0), EINVAL),
    (dict(q=P + 8), EALIGN), (dict(rope=P + 4), EALIGN), (dict(pos=P + 2), EALIGN),
    (dict(st=P + 1), EALIGN), (dict(qo=P + 2), EALIGN),
])
def test_kv_append_rope(o, expect):
    assert append(cache(), **o) == expect


def attn(c, **o):
    a = dict(q=P, qs=256, B=2, Q=1, Hq=4, pos=P, pre=P, plen=20, table=P, cols=4, mk=64, scale=0.1,
             out=P, lse=None, st=None, ws=P, wb=BIG)
    a.update(o)
    return moe.raw_call("attn_shared_prefix", c, a["q"], a["qs"], a["B"], a["Q"], a["Hq"],
                        a["pos"], a["pre"], a["plen"], a["table"], a["cols"], a["mk"], a["scale"],
                        a["out"], a["lse"], a["st"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("o,expect", [
    (dict(B=0), OK), (dict(B=0, ws=None, wb=0), OK), (dict(B=0, plen=0, pre=None), OK),
    (dict(B=0, mk=20, table=None, cols=0), OK),
    (dict(B=-1), EINVAL), (dict(Q=0), EINVAL), (dict(Hq=3), EINVAL), (dict(Hq=0), EINVAL),
    (dict(Hq=1026, qs=1 << 20), ENOTSUP), (dict(B=1 << 18, Q=2), ENOTSUP),
    (dict(B=1 << 17, Hq=1024, qs=1 << 16), ENOTSUP), (dict(q=None), EINVAL), (dict(pos=None), EINVAL),
    (dict(out=None), EINVAL), (dict(pre=None), EINVAL), (dict(plen=-1), EINVAL),
    (dict(plen=65), EINVAL), (dict(table=None), EINVAL), (dict(cols=3), EINVAL),
    (dict(mk=0), EINVAL), (dict(mk=65), EINVAL), (dict(mk=(1 << 28) + 1, cols=1 << 28), ENOTSUP),
    (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(qs=248), EINVAL), (dict(qs=257), EINVAL),
    (dict(q=P + 2), EALIGN), (dict(pos=P + 1), EALIGN), (dict(lse=P + 4), EALIGN),
    (dict(ws=None), EINVAL), (dict(ws=P + 16), EALIGN), (dict(wb=100), EWS),
])
def test_attn_shared_prefix(o, expect):
    assert attn(cache(), **o) == expect


def test_attn_workspace_is_enough_and_needed():
    n = moe._lib.attn_workspace_bytes(cache(), 2, 1, 4, 20, 64)
    assert n > 0 and attn(cache(), wb=n - 1) == EWS
    assert moe._lib.attn_workspace_bytes(cache(), 0, 1, 4, 20, 64) == 0
    assert moe._lib.attn_workspace_bytes(cache(), 2, 1, 3, 20, 64) == 0


def logprobs(**o):
    a = dict(z=P, dt=1, rs=100, T=3, V=100, tok=P, n=5, lp=P, ent=P, ids=P, tlp=P, st=None, ws=P,
             wb=BIG)
    a.update(o)
    return moe.raw_call("token_logprobs", a["z"], a["dt"], a["rs"], a["T"], a["V"], a["tok"],
                        a["n"], a["lp"], a["ent"], a["ids"], a["tlp"], a["st"], a["ws"], a["wb"],
                        None)


@pytest.mark.parametrize("o,expect", [
    (dict(T=0), OK), (dict(T=0, ws=None, wb=0), OK), (dict(T=0, tok=None, lp=None, ent=None), OK),
    (dict(T=0, n=0, ids=None, tlp=None), OK),
    (dict(z=None), EINVAL), (dict(dt=3), EINVAL), (dict(T=-1), EINVAL), (dict(V=0), EINVAL),
    (dict(T=(1 << 18) + 1), ENOTSUP), (dict(V=(1 << 24) + 1, rs=1 << 25), ENOTSUP),
    (dict(n=-1), EINVAL), (dict(n=65), ENOTSUP), (dict(V=4, n=5), EINVAL), (dict(rs=99), EINVAL),
    (dict(tok=None), EINVAL), (dict(lp=None), EINVAL), (dict(ids=None), EINVAL),
    (dict(tlp=None), EINVAL), (dict(z=P + 2), EALIGN), (dict(tok=P + 2), EALIGN),
    (dict(lp=P + 4), EALIGN), (dict(ws=None), EINVAL), (dict(ws=P + 16), EALIGN),
    (dict(wb=100), EWS),
])
def test_token_logprobs(o, expect):
    assert logprobs(**o) == expect


def test_token_logprobs_workspace():
    n = moe.token_logprobs_workspace_bytes(3, 100, 5)
    assert n > 0 and logprobs(wb=n - 1) == EWS
    assert moe.token_logprobs_workspace_bytes(0, 100, 5) == 0
    assert moe.token_logprobs_workspace_bytes(3, 100, 65) == 0
    assert moe.token_logprobs_workspace_bytes(3, 4, 5) == 0


def test_binding_raises():
    w = moe.make_w4(1, 64, 100, 32, P, P)
    with pytest.raises(moe.MoeError) as e:
        moe.w4_linear(w, P, 100, 1, P, 64, 2, stream=0)
    assert e.value.status == EINVAL
