"""logits_adjust against the rules in 64 bits; logits that no rule touches stay bit for bit."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"
DT = {"bf16": (moe.MOE_DT_BF16, torch.bfloat16), "f32": (moe.MOE_DT_F32, torch.float32)}
RULES = ("history", "seq_of", "n_tokens", "n_prompt", "repetition", "presence", "frequency", "bias_ids",
         "bias", "mask", "mask_of")


def run(rules, z, V, out_dt, pad_out=0, in_place=False, shift=0, stream=None):
    """rules: dict of CPU arrays; z [T][stride] CPU.  Returns out (CPU) and the status word.  shift: the
    buffers begin that many elements behind an aligned address."""
    T, zs = z.shape
    d = {k: torch.from_numpy(np.ascontiguousarray(rules[k])).to(DEV) for k in RULES if rules.get(k) is not None}
    kw = dict(d)
    if "history" in d:
        kw.update(history_stride=rules["history"].shape[1], n_seqs=rules["history"].shape[0],
                  max_history=rules.get("max_history", rules["history"].shape[1]))
    if "bias" in d:
        kw.update(n_bias=rules["bias"].shape[1])
    if "mask" in d:
        kw.update(mask_stride=rules["mask"].shape[1], n_masks=rules["mask"].shape[0])
    zb = torch.zeros(z.numel() + shift, dtype=z.dtype, device=DEV)
    zb[shift:] = z.reshape(-1).to(DEV)
    zd = zb[shift:].view(T, zs)
    os = zs if in_place else V + pad_out
    ob = torch.full((T * os + shift,), 9.0, dtype=DT[out_dt][1], device=DEV)
    o = zd if in_place else ob[shift:].view(T, os)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    zdt = moe.MOE_DT_BF16 if z.dtype == torch.bfloat16 else moe.MOE_DT_F32
    moe.logits_adjust(moe.make_logits_rules(**kw), zd, zdt, zs, T, V, o, DT[out_dt][0], os, st, stream)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(zd.cpu().view(torch.int16 if z.dtype == torch.bfloat16 else torch.int32),
                           z.view(torch.int16 if z.dtype == torch.bfloat16 else torch.int32))
        if pad_out:
            assert bool((o[:, V:] == 9).all())
    return o.cpu(), int(st.item())


def expect(rules, z, V):
    """In 64 bits: the values, the size of the terms, which logits a rule touched, the status."""
    T = z.shape[0]
    e = z[:, :V].double().numpy().copy()
    mag = np.abs(e)
    touched = np.zeros((T, V), bool)
    status = 0
    h = rules.get("history")
    top = rules.get("max_history", h.shape[1]) if h is not None else 0
    for t in range(T):
        if rules.get("bias") is not None:
            last = {}
            for i, b in zip(rules["bias_ids"][t], rules["bias"][t]):
                if i >= V:
                    status |= moe.MOE_STATUS_BAD_TOKEN
                elif i >= 0:
                    last[int(i)] = float(b)
            for i, b in last.items():
                e[t, i] += b
                mag[t, i] += abs(b)
                touched[t, i] = True
        if h is not None:
            seq = int(rules["seq_of"][t]) if rules.get("seq_of") is not None else t
            n = int(rules["n_tokens"][t])
            if seq >= h.shape[0] or (seq >= 0 and n > top):
                status |= moe.MOE_STATUS_BAD_INDEX
            text = h[seq, :max(0, min(n, top))] if 0 <= seq < h.shape[0] else np.zeros(0, int)
            given = int(rules["n_prompt"][t]) if rules.get("n_prompt") is not None else 0
            made = text[max(0, given):]
            if (text >= V).any():
                status |= moe.MOE_STATUS_BAD_TOKEN
            met = np.unique(text[(text >= 0) & (text < V)])
            touched[t, met] = True
            rep = float(rules["repetition"][t]) if rules.get("repetition") is not None else 1.0
            e[t, met] = np.where(e[t, met] > 0, e[t, met] / rep, e[t, met] * rep)
            mag[t, met] *= max(rep, 1 / rep)
            ids, c = np.unique(made[(made >= 0) & (made < V)], return_counts=True)
            p = float(rules["presence"][t]) if rules.get("presence") is not None else 0.0
            f = float(rules["frequency"][t]) if rules.get("frequency") is not None else 0.0
            e[t, ids] -= p + f * c
            mag[t, ids] += abs(p) + abs(f) * c
        if rules.get("mask") is not None:
            m = int(rules["mask_of"][t]) if rules.get("mask_of") is not None else t
            if m >= rules["mask"].shape[0]:
                status |= moe.MOE_STATUS_BAD_INDEX
            elif m >= 0:
                v = np.arange(V)
                off = (rules["mask"][m].view(np.uint32)[v // 32] >> (v % 32).astype(np.uint32)) & 1 == 0
                e[t, off] = -np.inf
                touched[t, off] = True
    return e, mag, touched, status


def check(rules, z, V, out_dt, **kw):
    got, st = run(rules, z, V, out_dt, **kw)
    e, mag, touched, status = expect(rules, z, V)
    assert st == status, (st, status)
    g = got[:, :V]
    same = z[:, :V].to(DT[out_dt][1])
    keep = torch.from_numpy(~touched)
    assert torch.equal(g[keep].view(torch.int16 if out_dt == "bf16" else torch.int32),
                       same[keep].view(torch.int16 if out_dt == "bf16" else torch.int32))
    gd = g.double().numpy()
    # a product past fp32's largest is an infinity in fp32
    e = np.where(np.abs(e) > np.finfo(np.float32).max, np.copysign(np.inf, e), e)
    fin = np.isfinite(e)
    assert np.array_equal(np.isfinite(gd), fin)
    assert np.array_equal(gd[~fin & ~np.isnan(e)], e[~fin & ~np.isnan(e)])
    assert np.array_equal(np.isnan(gd), np.isnan(e))
    # at most six fp32 operations, each off by 2^-24 of a term; then the output's rounding
    tol = 6 * 2.0 ** -24 * mag + (2.0 ** -8 if out_dt == "bf16" else 2.0 ** -24) * np.abs(np.where(fin, e, 0)) + 1e-40
    with np.errstate(invalid="ignore"):
        assert (np.abs(gd - e)[fin] <= tol[fin]).all(), np.abs(gd - e)[fin].max()


def rules_of(rng, T, V, L=0, nb=0, mask=False, prompt=True, seqs=None):
    r = {}
    if L:
        n = seqs or T
        r["history"] = np.minimum(V ** rng.random((n, L)) - 1, V - 1).astype(np.int32)
        r["n_tokens"] = rng.integers(0, L + 1, T).astype(np.int32)
        r["seq_of"] = rng.integers(0, n, T).astype(np.int32)
        if prompt:
            r["n_prompt"] = (r["n_tokens"] * rng.random(T)).astype(np.int32)
        r["repetition"] = (1 + 0.5 * rng.random(T)).astype(np.float32)
        r["presence"] = rng.random(T).astype(np.float32)
        r["frequency"] = (0.3 * rng.standard_normal(T)).astype(np.float32)
    if nb:
        r["bias_ids"] = rng.integers(-1, V, (T, nb)).astype(np.int32)
        r["bias"] = (3 * rng.standard_normal((T, nb))).astype(np.float32)
    if mask:
        n = max(1, T // 2)
        r["mask"] = rng.integers(-2 ** 31, 2 ** 31, (n, -(-V // 32) + 1)).astype(np.int32)
        r["mask_of"] = rng.integers(-1, n, T).astype(np.int32)
    return r


def logits(rng, T, stride, dt):
    return torch.from_numpy((3 * rng.standard_normal((T, stride))).astype(np.float32)).to(DT[dt][1])


@pytest.mark.parametrize("zdt,odt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("V", [1, 7, 33, 1000, 2048, 8191, 50021])
def test_all_rules(zdt, odt, V):
    rng = np.random.default_rng(V)
    for T, L, nb, mask in [(1, 5, 0, False), (3, 300, 4, True), (2, 0, 3, False), (5, 0, 0, True),
                           (4, 64, 0, True), (2, 0, 0, False), (17, 700, 30, True)]:
        print(V, zdt, odt, T, L, nb, mask, flush=True)
        z = logits(rng, T, V, zdt)
        r = rules_of(rng, T, V, L, nb, mask)
        check(r, z, V, odt)
        if zdt == odt:
            check(r, z, V, odt, in_place=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_rows_long_texts_and_odd_places(dt):
    """Blocks of 8192 ids; rows at every alignment of their elements; texts of 5000 tokens, of which
    some ids come thousands of times; several rows of one text."""
    rng = np.random.default_rng(5)
    T, V = 70, 16411
    z = logits(rng, T, V + 6, dt)
    r = rules_of(rng, T, V, 5000, 50, True, seqs=3)
    r["history"][0, ::2] = 8192
    for shift in (0, 1, 3):
        check(r, z, V, dt, pad_out=5, shift=shift)
        check(r, z, V, dt, in_place=True, shift=shift)


def test_partial_rules():
    """Each penalty alone, no prompt lengths, row's own text and mask (no indexes)."""
    rng = np.random.default_rng(6)
    T, V = 6, 777
    z = logits(rng, T, V, "f32")
    full = rules_of(rng, T, V, 90, 0, True)
    full["mask"] = np.repeat(full["mask"], 2, 0)
    for keep in (["repetition"], ["presence"], ["frequency"], []):
        r = {k: v for k, v in full.items() if k in ("history", "n_tokens") or k in keep}
        check(r, z, V, "f32")
    check({"mask": full["mask"]}, z, V, "f32")


def test_special_logits_and_masks_that_leave_nothing():
    rng = np.random.default_rng(7)
    T, V = 5, 300
    z = logits(rng, T, V, "f32")
    z[0, 3], z[0, 4], z[0, 5] = float("nan"), float("inf"), float("-inf")
    z[1, :] = torch.finfo(torch.float32).min
    r = rules_of(rng, T, V, 0, 0, True)
    r["mask"] = np.zeros((2, 10), np.int32)
    r["mask"][1] = -1
    r["mask_of"] = np.array([0, 1, 0, 1, -1], np.int32)      # all masked: also NaN and +inf
    check(r, z, V, "f32")
    got, _ = run(r, z, V, "f32")
    assert bool((got[0] == -np.inf).all()) and bool((got[2] == -np.inf).all())
    # a NaN that is allowed stays one, under penalties too
    r = {"history": np.array([[3, 4, 5, 3]] * 5, np.int32), "n_tokens": np.full(5, 4, np.int32),
         "repetition": np.full(5, 1.5, np.float32), "presence": np.full(5, 1.0, np.float32)}
    check(r, z, V, "f32")


def test_several_entries_of_one_id():
    """The last entry of an id counts, whatever its neighbours; a negative id is none."""
    T, V = 2, 40
    z = torch.zeros((T, V))
    ids = np.array([[5, 5, -1, 7, 5, 7], [0, 39, 0, 39, 0, 39]], np.int32)
    b = np.array([[1, 2, 3, 4, 5, 6], [1, 2, 3, 4, 5, 6]], np.float32)
    got, st = run({"bias_ids": ids, "bias": b}, z, V, "f32")
    want = torch.zeros((T, V))
    want[0, 5], want[0, 7], want[1, 0], want[1, 39] = 5, 6, 5, 6
    assert torch.equal(got, want) and st == 0


def test_indexes_out_of_range_are_reported_and_left_out():
    rng = np.random.default_rng(8)
    T, V = 4, 100
    z = logits(rng, T, V, "f32")
    base = rules_of(rng, T, V, 20, 3, True)
    for key, at, val in [("history", (0, 0), V), ("history", (1, 3), 2 ** 31 - 1), ("history", (0, 1), -5),
                         ("seq_of", 2, 4), ("seq_of", 1, -3), ("n_tokens", 0, 21), ("n_tokens", 1, -4),
                         ("n_prompt", 0, 99), ("n_prompt", 0, -99), ("bias_ids", (2, 1), V), ("bias_ids", (0, 0), -9),
                         ("mask_of", 3, 2), ("mask_of", 3, -2 ** 31)]:
        r = {k: v.copy() for k, v in base.items()}
        r["n_tokens"][:] = 20
        r["seq_of"][:] = np.arange(T)
        r[key][at] = val
        print(key, at, val, flush=True)
        check(r, z, V, "f32")
    r = {k: v.copy() for k, v in base.items()}
    r["max_history"] = 7                      # shorter than the rows
    check(r, z, V, "f32")


def test_captured_beside_eager_calls():
    rng = np.random.default_rng(9)
    T, V = 9, 20011
    r = rules_of(rng, T, V, 200, 5, True)
    d = {k: torch.from_numpy(v).to(DEV) for k, v in r.items()}
    z = logits(rng, T, V, "f32")
    zd, o = z.to(DEV), torch.empty((T, V), device=DEV)
    rules = moe.make_logits_rules(history_stride=200, n_seqs=T, max_history=200, n_bias=5,
                                  mask_stride=r["mask"].shape[1], n_masks=r["mask"].shape[0], **d)

    def go(out):
        moe.logits_adjust(rules, zd, moe.MOE_DT_F32, V, T, V, out, moe.MOE_DT_F32, V, None)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        go(o)
    for i in range(3):
        zd.copy_(logits(rng, T, V, "f32"))
        d["n_tokens"].copy_(torch.randint(0, 201, (T,)))
        e = torch.empty_like(o)
        go(e)
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view(torch.int32), e.view(torch.int32))


@pytest.mark.parametrize("zdt,odt", [("bf16", "f32"), ("f32", "bf16")])
def test_blocks_of_8192_ids_into_the_other_type(zdt, odt):
    rng = np.random.default_rng(11)
    T, V = 70, 16411
    z = logits(rng, T, V, zdt)
    r = rules_of(rng, T, V, 900, 20, True, seqs=3)
    for shift in (0, 1):
        check(r, z, V, odt, pad_out=3, shift=shift)


@pytest.mark.parametrize("dt,in_place", [("f32", False), ("bf16", False), ("f32", True), ("bf16", True)])
def test_rows_past_the_grids_own(dt, in_place):
    """More rows than a grid has (32768): its blocks take several, each with that row's own rules."""
    rng = np.random.default_rng(5)
    T, V = 32768 + 517, 67
    z = torch.from_numpy((3 * rng.standard_normal((T, V))).astype(np.float32)).to(DT[dt][1])
    r = rules_of(rng, T, V, L=9, nb=2, mask=True, seqs=700)
    r["seq_of"][32768:] = rng.permutation(700)[:517]
    check(r, z, V, dt, in_place=in_place)
    check({k: v for k, v in r.items() if k.startswith("mask")}, z, V, dt, in_place=in_place)
    r["bias_ids"][32768, 0], r["seq_of"][33000], r["mask_of"][T - 1] = V, 700, r["mask"].shape[0]
    check(r, z, V, dt, in_place=in_place)
