"""CPU tests of the argument checks of add_rmsnorm, lora_linear and logits_adjust: every refusal
happens on the host before any HIP call (no GPU needed), and empty batches are accepted without a
device."""
import ctypes
import os
import subprocess

import pytest

moe = pytest.importorskip("bit_expert_ffn_moe_amd")

P, BIG = 0x100000, 1 << 40
EINVAL, ENOTSUP, EALIGN, EWS, OK = (moe.MOE_EINVAL, moe.MOE_ENOTSUP, moe.MOE_EALIGN,
                                    moe.MOE_EWORKSPACE, moe.MOE_OK)


def norm(**o):
    a = dict(x=P, xs=256, res=P, dt=1, rs=256, T=3, H=256, w=P, eps=1e-6, ro=P, y=P, q=P, s=P)
    a.update(o)
    return moe.raw_call("add_rmsnorm", a["x"], a["xs"], a["res"], a["dt"], a["rs"], a["T"], a["H"],
                        a["w"], a["eps"], a["ro"], a["y"], a["q"], a["s"], None)


@pytest.mark.parametrize("o,expect", [
    (dict(T=0), OK), (dict(T=0, res=None, ro=None, dt=0, rs=0), OK), (dict(T=0, w=None), OK),
    (dict(T=0, q=None, s=None, H=8), OK), (dict(T=0, y=None), OK), (dict(T=0, dt=2), OK),
    (dict(T=0, ro=None), OK),
    (dict(x=None), EINVAL), (dict(y=None, q=None, s=None), EINVAL), (dict(q=None), EINVAL),
    (dict(s=None), EINVAL), (dict(res=None), EINVAL), (dict(dt=3), EINVAL), (dict(T=-1), EINVAL),
    (dict(H=0), EINVAL), (dict(H=132), EINVAL), (dict(H=136), EINVAL), (dict(xs=248), EINVAL),
    (dict(xs=260), EINVAL), (dict(rs=248), EINVAL), (dict(rs=257), EINVAL), (dict(eps=0.0), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(eps=2.0 ** -101), EINVAL), (dict(T=0, eps=2.0 ** -100), OK),
    (dict(T=(1 << 18) + 1), ENOTSUP), (dict(H=16512, xs=16512, rs=16512), ENOTSUP),
    (dict(x=P + 8), EALIGN), (dict(res=P + 2), EALIGN), (dict(w=P + 8), EALIGN),
    (dict(ro=P + 4), EALIGN), (dict(y=P + 8), EALIGN), (dict(q=P + 8), EALIGN),
    (dict(s=P + 4), EALIGN),
])
def test_add_rmsnorm(o, expect):
    assert norm(**o) == expect


def adapters(**o):
    a = dict(n=4, R=16, K=128, N=100, a=P, b=P, rank=None, scale=None)
    a.update(o)
    return ctypes.byref(moe.make_lora(a["n"], a["R"], a["K"], a["N"], a["a"], a["b"], a["rank"], a["scale"]))


def lora(w, **o):
    a = dict(x=P, xs=128, T=3, of=P, base=P, bs=100, y=2 * P, ys=100, dt=1, st=None, ws=P, wb=BIG)
    a.update(o)
    return moe.raw_call("lora_linear", w, a["x"], a["xs"], a["T"], a["of"], a["base"], a["bs"], a["y"],
                        a["ys"], a["dt"], a["st"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("w,expect", [
    (dict(n=0), EINVAL), (dict(R=0), EINVAL), (dict(R=12), EINVAL), (dict(K=0), EINVAL),
    (dict(K=100), EINVAL), (dict(N=0), EINVAL), (dict(a=None), EINVAL), (dict(b=None), EINVAL),
    (dict(n=65537), ENOTSUP), (dict(R=136), ENOTSUP), (dict(K=(1 << 20) + 8), ENOTSUP),
    (dict(N=(1 << 20) + 1), ENOTSUP), (dict(a=P + 8), EALIGN), (dict(b=P + 2), EALIGN),
    (dict(rank=P + 2), EALIGN), (dict(scale=P + 1), EALIGN),
])
def test_bad_adapters(w, expect):
    assert lora(adapters(**w)) == expect
    assert moe._lib.lora_workspace_bytes(adapters(**w), 3) == 0


@pytest.mark.parametrize("o,expect", [
    (dict(T=0), OK), (dict(T=0, ws=None, wb=0), OK), (dict(T=0, base=None, bs=0), OK),
    (dict(T=0, base=2 * P), OK), (dict(T=0, dt=2), OK),
    (dict(x=None), EINVAL), (dict(of=None), EINVAL), (dict(y=None), EINVAL), (dict(T=-1), EINVAL),
    (dict(dt=3), EINVAL), (dict(xs=120), EINVAL), (dict(xs=132), EINVAL), (dict(ys=99), EINVAL),
    (dict(bs=99), EINVAL), (dict(base=2 * P, bs=104), EINVAL), (dict(T=(1 << 18) + 1), ENOTSUP),
    (dict(x=P + 8), EALIGN), (dict(base=P + 2), EALIGN), (dict(y=P + 4), EALIGN),
    (dict(of=P + 2), EALIGN), (dict(st=P + 1), EALIGN), (dict(ws=None), EINVAL),
    (dict(ws=P + 16), EALIGN), (dict(wb=100), EWS),
])
def test_lora_linear(o, expect):
    assert lora(adapters(), **o) == expect


def test_lora_null_descriptor_and_workspace():
    assert lora(None) == EINVAL
    n = moe._lib.lora_workspace_bytes(adapters(), 3)
    assert n > 0 and lora(adapters(), wb=n - 1) == EWS
    assert moe._lib.lora_workspace_bytes(adapters(), 0) == 0
    assert moe._lib.lora_workspace_bytes(adapters(), (1 << 18) + 1) == 0


@pytest.mark.parametrize("K", [128, 4096, 8192, 16384, 20000, 1 << 20])
@pytest.mark.parametrize("R", [8, 32, 128])
def test_lora_workspace_of_a_batch_holds_every_smaller_one(R, K):
    """Parts of x's columns get fewer as tokens get more; the bytes never do."""
    w = adapters(R=R, K=K)
    before = 0
    for T in [*range(1, 1020, 7), *range(1020, 17000), 1 << 17, 1 << 18]:
        n = moe._lib.lora_workspace_bytes(w, T)
        assert n >= before, (T, n, before)
        before = n


FULL = dict(history=P, history_stride=50, max_history=50, n_seqs=3, seq_of=P, n_tokens=P, n_prompt=P,
            repetition=P, presence=P, frequency=P, bias_ids=P, bias=P, n_bias=4, mask=P, mask_stride=4,
            n_masks=2, mask_of=P)


def logits(rules, **o):
    r = dict(FULL)
    r.update(rules)
    a = dict(z=P, zd=2, zs=100, T=3, V=100, out=2 * P, od=2, os=100, st=None)
    a.update(o)
    return moe.raw_call("logits_adjust", ctypes.byref(moe.make_logits_rules(**r)), a["z"], a["zd"],
                        a["zs"], a["T"], a["V"], a["out"], a["od"], a["os"], a["st"], None)


NO_HISTORY = dict(history=None, repetition=None, presence=None, frequency=None)


@pytest.mark.parametrize("rules,call,expect", [
    ({}, dict(T=0), OK), (NO_HISTORY, dict(T=0), OK), ({}, dict(T=0, out=P), OK),
    (dict(bias=None, bias_ids=None, n_bias=0), dict(T=0), OK), (dict(mask=None), dict(T=0), OK),
    (dict(seq_of=None, n_prompt=None, mask_of=None), dict(T=0), OK), ({}, dict(T=0, od=1), OK),
    ({}, dict(T=0, z=P + 4, out=2 * P + 4), OK),
    ({}, dict(z=None), EINVAL), ({}, dict(out=None), EINVAL), ({}, dict(zd=3), EINVAL),
    ({}, dict(od=0), EINVAL), ({}, dict(T=-1), EINVAL), ({}, dict(V=0), EINVAL),
    ({}, dict(zs=99), EINVAL), ({}, dict(os=99), EINVAL), ({}, dict(out=P, od=1), EINVAL),
    ({}, dict(out=P, os=101), EINVAL),
    (dict(n_tokens=None), {}, EINVAL), (dict(n_seqs=0), {}, EINVAL), (dict(max_history=0), {}, EINVAL),
    (dict(max_history=51), {}, EINVAL), (dict(history=None), {}, EINVAL),
    (dict(n_bias=-1), {}, EINVAL), (dict(n_bias=0), {}, EINVAL), (dict(bias=None), {}, EINVAL),
    (dict(bias_ids=None), {}, EINVAL), (dict(n_masks=0), {}, EINVAL), (dict(mask_stride=3), {}, EINVAL),
    ({}, dict(T=(1 << 18) + 1), ENOTSUP),
    (dict(mask=None), dict(V=(1 << 24) + 1, zs=1 << 25, os=1 << 25), ENOTSUP),
    (dict(max_history=1 << 20, history_stride=1 << 20), {}, ENOTSUP), (dict(n_bias=2048), {}, ENOTSUP),
    ({}, dict(z=P + 2), EALIGN), ({}, dict(zd=1, z=P + 1), EALIGN), ({}, dict(out=P + 2), EALIGN),
    ({}, dict(st=P + 2), EALIGN),
] + [({k: P + 2}, {}, EALIGN) for k in ("history", "seq_of", "n_tokens", "n_prompt", "repetition",
                                        "presence", "frequency", "bias_ids", "bias", "mask", "mask_of")])
def test_logits_adjust(rules, call, expect):
    assert logits(rules, **call) == expect


def test_logits_null_rules_and_binding_errors():
    assert moe.raw_call("logits_adjust", None, P, 2, 100, 3, 100, 2 * P, 2, 100, None, None) == EINVAL
    with pytest.raises(moe.MoeError) as e:
        moe.add_rmsnorm(P, 128, None, 0, 0, 1, 100, None, 1e-6, None, P, None, None, stream=0)
    assert e.value.status == EINVAL
    w = moe.make_lora(1, 12, 64, 64, P, P)
    with pytest.raises(moe.MoeError):
        moe.lora_linear(w, P, 64, 1, P, None, 0, P, 64, 1, None, P, BIG, stream=0)
    with pytest.raises(moe.MoeError):
        moe.logits_adjust(moe.make_logits_rules(), P, 1, 9, 1, 10, P, 1, 10, None, stream=0)


def test_a_cache_in_4_bits_has_its_scales():
    def rc(**o):
        a = dict(dt=4, n=10, page=16, Hkv=2, D=64, k=P, v=P, ks=P, vs=P)
        a.update(o)
        c = ctypes.byref(moe.make_kv_cache(a["dt"], a["n"], a["page"], a["Hkv"], a["D"], a["k"], a["v"],
                                           a["ks"], a["vs"]))
        app = moe.raw_call("kv_append_rope", c, P, 256, 4, P, 128, P, 128, 0, None, 0, 0, 0, P, P, P, 2, 4,
                           P, None, None)
        att = moe.raw_call("attn_shared_prefix", c, P, 256, 0, 1, 4, P, P, 20, P, 4, 64, 0.1, P, None,
                           None, None, 0, None)
        assert app == att
        assert (moe._lib.attn_workspace_bytes(c, 2, 1, 4, 20, 64) > 0) == (app == OK)
        return app
    assert rc() == OK
    assert rc(ks=None) == EINVAL and rc(vs=None) == EINVAL and rc(dt=5) == EINVAL
    assert rc(ks=P + 8) == EALIGN and rc(D=96) == ENOTSUP and rc(page=8) == ENOTSUP


@pytest.mark.parametrize("shared,own,parts", [(10000, 41000, 8 + 23), (2000, 9000, 4 + 24), (0, 9000, 24)])
def test_blocks_of_32_rows_of_its_own_keys_are_the_prefixs_too(shared, own, parts):
    """One sequence of 16 tokens, 8 kv heads of 8 query heads, 128 columns: 128 rows over shared E2M1 keys and many
    of its own, which blocks of 32 rows take.  The shared keys are cut for 8 heads x 4 such blocks and a
    block a CU (few of them: a block for two), the own for the three blocks a CU that are left.  Each
    part leaves a row's maximum, sum and columns."""
    c = ctypes.byref(moe.make_kv_cache(4, 1000, 16, 8, 128, P, P, P, P))
    rows = 16 * 64
    assert moe._lib.attn_workspace_bytes(c, 1, 16, 64, shared, shared + own) == parts * rows * (8 + 4 * 128)


@pytest.mark.parametrize("cc", [["gcc", "-xc", "-std=c99"], ["g++", "-xc++", "-std=c++11"]])
def test_programs_written_for_an_e4m3_cache_compile(cc):
    """The scales of a cache descriptor are floats to read and write, without a cast."""
    src = b"""#include "moe.h"
static float row_scale(const kv_cache* c, int64_t row) { float* s = c->k_scale; return s[row] * c->v_scale[row]; }
float use(float* k, float* v) {
  kv_cache c = {MOE_DT_FP8_E4M3, 1, 16, 1, 64, 0, k, v, k, v};
  c.k_scale = k;
  return row_scale(&c, 0);
}
"""
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    r = subprocess.run([*cc, "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I", inc, "-"], input=src,
                       capture_output=True, timeout=60)
    assert r.returncode == 0, r.stderr.decode()


@pytest.mark.parametrize("V", [1, 1000, 50021, 1 << 24])
@pytest.mark.parametrize("n", [0, 1, 64])
def test_logprobs_workspace_of_a_batch_holds_every_smaller_one(V, n):
    """Many rows need no partial results, some smaller batches do; the bytes never fall."""
    if n > V:
        pytest.skip("more than there are")
    before = 0
    for T in [*range(1, 700), 1000, 1 << 14, 1 << 18]:
        b = moe._lib.token_logprobs_workspace_bytes(T, V, n)
        assert b >= before, (T, b, before)
        before = b
