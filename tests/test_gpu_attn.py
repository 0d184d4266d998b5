"""attn_shared_prefix against attention in 64 bits.

Tolerance of an output: probabilities rounded to bf16 (8 significant bits, so
half a unit is up to 2^-8 of the value) move it by at most 2^-8 sum p|v|, its own
rounding by 2^-8 |o|; an fp32 score is off by at most
d = 2 D 2^-23 sum |q k| scale, which moves every probability by 2 d at most; 5% and
2^-16 sum p|v| are for the fp32 sums.  lse: d and 8 units of fp32."""
import numpy as np
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


def build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8):
    """A cache with B sequences of own[b] keys after P shared ones, and random
    queries.  The page holding key P is private to each sequence."""
    n_max = P + max(own)
    cols, shared = -(-n_max // page), P // page
    n_pre = -(-P // page)
    n_pages = n_pre + B * (cols - shared) + 2
    perm = rng.permutation(n_pages)
    pre = perm[:n_pre]
    mine = perm[n_pre:n_pre + B * (cols - shared)].reshape(B, cols - shared)
    table = np.concatenate([np.full((B, shared), -99), mine], 1)  # the prefix's entries: not read
    kv = ref.Cache(rng, n_pages, page, Hkv, D, fp8)
    q = ref.bf16(2 * rng.standard_normal((B * Q, Hq, D)).astype(np.float32))
    return kv, q, pre, table, n_max


def call(kv, q, pos, pre, P, table, max_keys, scale, Q, extra=0, expect_status=0, stream=None):
    T, Hq, D = q.shape
    B = T // Q
    d = {n: t.to(DEV) if t is not None else None for n, t in kv.t.items()}
    n_pages, Hkv, page = d["k"].shape[:3]
    c = moe.make_kv_cache(moe.MOE_DT_FP8_E4M3 if kv.fp8 else moe.MOE_DT_BF16, n_pages, page, Hkv, D,
                          d["k"], d["v"], d["ks"], d["vs"])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    qd = torch.full((T, Hq * D + extra), float("nan"), dtype=torch.bfloat16)
    qd[:, :Hq * D] = q.reshape(T, -1)
    qd = qd.to(DEV)
    nb = moe.attn_workspace_bytes(c, B, Q, Hq, P, max_keys)
    assert nb > 0
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)   # NaN where nothing is written
    out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 9.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos_d, pre_d, table_d = i32(pos), i32(pre) if P else None, i32(table)
    moe.attn_shared_prefix(c, qd, Hq * D + extra, B, Q, Hq, pos_d, pre_d, P, table_d,
                           table.shape[1], max_keys, scale, out, lse, st, ws, nb, stream)
    torch.cuda.synchronize()
    assert int(st.item()) == expect_status
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def check(o, lse, q, kv, pos, pre, P, table, scale, Q, max_keys):
    eo, el, mag, qk = ref.attention(q.double().numpy(), kv, pos, pre, P, table, scale, Q, max_keys)
    d = 2 * q.shape[2] * 2.0 ** -23 * qk
    tol = 1.05 * 2.0 ** -8 * (mag + np.abs(eo)) + (2 * d[..., None] + 2.0 ** -16) * mag
    assert (np.abs(o - eo) <= tol).all(), np.nanmax(np.abs(o - eo) / (tol + 1e-300))
    none = el == -np.inf
    assert np.array_equal(lse == -np.inf, none)
    assert (np.abs(lse - el)[~none] <= (d + 2.0 ** -20 * (1 + np.abs(el)))[~none]).all()
    assert (o[none] == 0).all()


def positions(own, P, Q):
    """The last of Q tokens of sequence b sees P + own[b] keys; own[b] < 0: padding."""
    return np.array([P + n - Q + i if n >= 0 else -1 for n in own for i in range(Q)])


SHAPES = [  # B, Q, Hq, Hkv, D, page, P, own
    (1, 1, 1, 1, 64, 16, 0, [1]),                     # one key in all
    (1, 1, 1, 1, 128, 16, 1, [1]),
    (3, 1, 4, 4, 64, 16, 0, [5, 16, 33]),             # no prefix, one head per kv head
    (2, 1, 8, 1, 128, 32, 40, [1, 70]),               # one kv head, prefix ends in a page
    (4, 1, 14, 2, 64, 16, 500, [60, 1, -1, 17]),      # 7 heads a group, an empty sequence
    (2, 4, 8, 2, 128, 64, 129, [4, 200]),             # four tokens a sequence
    (3, 3, 12, 4, 256, 32, 95, [3, 64, 65]),
    (5, 2, 32, 8, 128, 128, 300, [2, 129, 700, 300, 31]),
    (20, 1, 8, 2, 64, 16, 333, list(range(1, 21))),   # more rows than a tile
    (2, 40, 3, 1, 64, 16, 50, [40, 90]),              # a prompt's chunk of 40 tokens
    (1, 1, 2, 1, 128, 1024, 1500, [600]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_64_bit_attention(shape, fp8):
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, fp8, flush=True)
    rng = np.random.default_rng(B * 100 + P)
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    pos = positions(own, P, Q)
    scale = D ** -0.5
    for max_keys in (n, table.shape[1] * page):
        o, lse = call(kv, q, pos, pre, P, table, max_keys, scale, Q, extra=8)
        check(o, lse, q, kv, pos, pre, P, table, scale, Q, max_keys)


@pytest.mark.parametrize("fp8", [False, True])
def test_long_axes_are_split(fp8):
    rng = np.random.default_rng(4)
    B, Q, Hq, Hkv, D, page, P, own = 2, 1, 4, 1, 128, 64, 5000, [3000, 1234]
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    pos = positions(own, P, Q)
    o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_that_see_part_of_the_prefix_or_nothing(fp8):
    """Limits inside the prefix, at its end, and empty rows among full ones."""
    rng = np.random.default_rng(5)
    B, Q, Hq, Hkv, D, page, P = 6, 2, 4, 2, 64, 16, 70
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, [50] * B, fp8)
    pos = np.array([-1, -1, 0, 5, 68, 69, 70, 71, -1, 119, 31, 32])
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    check(o, lse, q, kv, pos, pre, P, table, 0.125, Q, n)
    # all rows empty
    o, lse = call(kv, q, np.full(12, -1), pre, P, table, n, 0.125, Q)
    assert (o == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_what_a_row_does_not_see_does_not_enter(fp8, bad):
    """NaN or inf in K, V (and scales) at every key past a row's limit, the free
    part of pages, and the private page's slots before the prefix's end."""
    rng = np.random.default_rng(6)
    B, Q, Hq, Hkv, D, page, P = 3, 3, 4, 2, 64, 32, 45
    own = [9, 40, 64]
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, own, fp8)
    pos = positions(own, P, Q)
    pos[2] = 20                       # one row ends inside the prefix
    seen = {(b, j) for b in range(B) for j in range(max(pos[b * Q:(b + 1) * Q]) + 1)}
    clean, lse_c = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    check(clean, lse_c, q, kv, pos, pre, P, table, 0.125, Q, n)
    val = float(bad)
    used = {(int(pre[j // page]), j % page) for j in range(P)} | \
        {(int(table[b, j // page]), j % page) for b, j in seen if j >= P}
    for pg in range(kv.t["k"].shape[0]):
        for s in range(page):
            if (pg, s) in used:
                continue
            if fp8:
                kv.t["k"][pg, :, s] = kv.t["v"][pg, :, s] = 0x7F
                kv.t["ks"][pg, :, s] = kv.t["vs"][pg, :, s] = val
            else:
                kv.t["k"][pg, :, s] = kv.t["v"][pg, :, s] = val
    # keys that the sequence's last row sees and its first ones do not
    for b in range(B):
        j = pos[b * Q + 2] if b else pos[1]
        pg, s = int(table[b, j // page]), j % page
        if fp8:
            kv.t["v"][pg, :, s] = 0x7F
            kv.t["vs"][pg, :, s] = val
        else:
            kv.t["v"][pg, :, s] = val
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    dirty = {1} | {b * Q + 2 for b in range(1, B)}
    for t in range(B * Q):
        if t in dirty:
            assert not np.isfinite(o[t]).any(), t
        else:
            assert np.array_equal(o[t], clean[t]) and np.array_equal(lse[t], lse_c[t]), t


def test_nan_in_the_prefix_past_a_short_row():
    rng = np.random.default_rng(7)
    B, Q, Hq, Hkv, D, page, P = 2, 1, 2, 1, 128, 16, 200
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, [5, 5], False)
    pos = np.array([100, 204])
    clean, _ = call(kv, q, pos, pre, P, table, n, 0.1, Q)
    kv.t["v"][int(pre[150 // page]), :, 150 % page] = float("inf")
    o, _ = call(kv, q, pos, pre, P, table, n, 0.1, Q)
    assert np.array_equal(o[0], clean[0]) and not np.isfinite(o[1]).any()


def test_large_scores_and_minus_infinity():
    """Scores of hundreds, a key of -inf (probability 0) and a row with
    nothing but such keys (as an empty row)."""
    rng = np.random.default_rng(8)
    B, Q, Hq, Hkv, D, page, P = 2, 1, 1, 1, 64, 16, 20
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, [30, 30], False)
    q = (q.float() * 40).to(torch.bfloat16)
    pos = positions([30, 30], P, Q)
    o, lse = call(kv, q, pos, pre, P, table, n, 1.0, Q)
    check(o, lse, q, kv, pos, pre, P, table, 1.0, Q, n)
    q[0, :, 0] = 1.0
    kv.t["k"][int(pre[0]), :, 3, 0] = -float("inf")
    q[1, :, 0] = 1.0
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    check(o, lse, q, kv, pos, pre, P, table, 0.125, Q, n)
    kv.t["k"][:, :, :, 0] = -float("inf")
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_bad_pages_and_bounds_are_reported():
    rng = np.random.default_rng(9)
    B, Q, Hq, Hkv, D, page, P = 2, 1, 4, 2, 64, 16, 40
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, [60, 20], False)
    pos = positions([60, 20], P, Q)
    table[0, 3] = 10 ** 6
    o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)
    pre = pre.copy()
    pre[1] = -1
    o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)
    # a token past max_keys sees the keys below it
    kv, q, pre, table, n = build(rng, B, Q, Hq, Hkv, D, page, P, [60, 20], False)
    o, lse = call(kv, q, pos, pre, P, table, 70, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
    check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, 70)


def test_repeatable_and_on_another_stream():
    rng = np.random.default_rng(10)
    kv, q, pre, table, n = build(rng, 4, 1, 8, 2, 128, 64, 600, [100, 200, 300, 400], False)
    pos = positions([100, 200, 300, 400], 600, 1)
    a = call(kv, q, pos, pre, 600, table, n, 0.1, 1)
    b = call(kv, q, pos, pre, 600, table, n, 0.1, 1, stream=torch.cuda.Stream())
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_cache_past_4_gib():
    """Keys and values in the last pages of a cache of over 4 GiB."""
    Hkv, D, page = 8, 128, 64
    n_pages = (1 << 32) // (Hkv * D * page * 2) + 4
    k = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    k[-2:] = torch.randn(k[-2:].shape, device=DEV).to(torch.bfloat16)
    v[-2:] = torch.randn(v[-2:].shape, device=DEV).to(torch.bfloat16)
    c = moe.make_kv_cache(moe.MOE_DT_BF16, n_pages, page, Hkv, D, k, v)
    q = torch.randn((1, Hkv, D), device=DEV).to(torch.bfloat16)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([127], dtype=torch.int32, device=DEV)
    nb = moe.attn_workspace_bytes(c, 1, 1, Hkv, 0, 128)
    ws, o = torch.empty(nb, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    moe.attn_shared_prefix(c, q, Hkv * D, 1, 1, Hkv, pos, None, 0, table, 2, 128, 0.1, o, None,
                           None, ws, nb)
    kk = torch.cat([k[-1], k[-2]], 1).double().cpu()
    vv = torch.cat([v[-1], v[-2]], 1).double().cpu()
    p = torch.softmax((kk * q[0].double().cpu()[:, None]).sum(-1) * 0.1, -1)
    want = (p[..., None] * vv).sum(1)
    mag = (p[..., None] * vv.abs()).sum(1)
    err = (o[0].double().cpu() - want).abs()
    assert (err <= 1.05 * 2.0 ** -8 * (mag + want.abs()) + 2.0 ** -12 * mag).all()
