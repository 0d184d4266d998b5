"""The key/value cache in 4 bits (E2M1 codes, a power of two per 32 columns): kv_append_rope into it
bit for bit against the rule, attn_shared_prefix over it against 64 bits at the shapes of the other
types.  The cache's values are bf16 values, so attention's tolerances are those of test_gpu_attn."""
import numpy as np
import pytest
import torch

import ops_ref as ref
from test_gpu_attn import SHAPES as FEW, build, check, positions
from test_gpu_attn_shapes import MANY, SHAPES, compare

pytestmark = pytest.mark.gpu

import bit_expert_ffn_moe_amd as moe  # noqa: E402

# beside the other types' shapes: rows enough (over 512 of a kv head) for key tiles in LDS at 64 and 128
# columns, for the shared keys, a sequence's own and both
TILES = [
    (5, 40, 16, 2, 128, 16, 300, [40, 64, 150, 90, 77]),
    (2, 600, 2, 2, 64, 32, 100, [600, 700]),
    (1, 520, 1, 1, 128, 64, 0, [777]),
    (66, 4, 8, 4, 64, 128, 130, [4 + i % 7 for i in range(66)]),
]

DEV = "cuda:0"
FP4 = moe.MOE_DT_FP4_E2M1
MAG = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def fp4_rows(x):
    """Codes [..., D/2] and scale bytes [..., D/32] (uint8) of float32 rows: the definition, group by
    group in float64."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(g).max(-1)
    none = ~np.isfinite(g).all(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.where(amax > 0, np.ceil(np.log2(np.where(none | (amax == 0), 1.0, amax) / 6.0)), -127)
        # the logarithm may be off by a unit beside a power of two
        e = np.where(amax <= 6 * 2.0 ** (e - 1), e - 1, e)
        e = np.where(amax > 6 * 2.0 ** e, e + 1, e)
    e = np.clip(e, -127, 125)
    u = np.where(none[..., None], 0.0, np.abs(g) / 2.0 ** e[..., None])
    # nearest, ties to the even code
    d = np.abs(u[..., None] - MAG)
    best = d.min(-1, keepdims=True)
    near = d == best
    code = np.argmax(near, -1)
    other = 7 - np.argmax(near[..., ::-1], -1)
    code = np.where(code % 2 == 0, code, other).astype(np.uint8)
    code |= np.where(np.signbit(g) & ~none[..., None], 8, 0).astype(np.uint8)
    code = code.reshape(x.shape)
    sb = np.where(none, 255, e + 127).astype(np.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, sb


class Cache4:
    """As ops_ref.Cache, in 4 bits."""

    def __init__(self, kv):
        self.page, self.t = kv.page, {}
        for n in "kv":
            codes, sb = fp4_rows(kv.values(n).astype(np.float32))
            self.t[n], self.t[n + "s"] = torch.from_numpy(codes), torch.from_numpy(sb)

    def values(self, n):
        b = self.t[n].numpy()
        x = np.empty((*b.shape[:-1], 2 * b.shape[-1]))
        x[..., 0::2], x[..., 1::2] = ref.E2M1[b & 15], ref.E2M1[b >> 4]
        s = self.t[n + "s"].numpy()
        f = np.where(s > 252, np.nan, np.ldexp(1.0, s.astype(int) - 127))
        return x * np.repeat(f, 32, -1)


def build4(rng, *shape):
    kv, q, pre, table, n = build(rng, *shape, False)
    return Cache4(kv), q, pre, table, n


def call(kv, q, pos, pre, P, table, max_keys, scale, Q, extra=0, expect_status=0, stream=None):
    T, Hq, D = q.shape
    B = T // Q
    d = {n: t.to(DEV) for n, t in kv.t.items()}
    n_pages, Hkv, page = d["k"].shape[:3]
    c = moe.make_kv_cache(FP4, n_pages, page, Hkv, D, d["k"], d["v"], d["ks"], d["vs"])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    qd = torch.full((T, Hq * D + extra), float("nan"), dtype=torch.bfloat16)
    qd[:, :Hq * D] = q.reshape(T, -1)
    qd = qd.to(DEV)
    nb = moe.attn_workspace_bytes(c, B, Q, Hq, P, max_keys)
    assert nb > 0
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, Hq), 9.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    pos_d, pre_d, table_d = i32(pos), i32(pre) if P else None, i32(table)
    moe.attn_shared_prefix(c, qd, Hq * D + extra, B, Q, Hq, pos_d, pre_d, P, table_d,
                           table.shape[1], max_keys, scale, out, lse, st, ws, nb, stream)
    torch.cuda.synchronize()
    assert int(st.item()) == expect_status
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


# ---- append -----------------------------------------------------------------------

def append(x, T, Hq, Hkv, D, page, rot, pairs, seq, pos, table, n_pages, extra=0, status=0):
    """kv_append_rope of x [T][(Hq + 2 Hkv) D + extra] bf16 into a cache of random bytes; compares
    everything it may and may not write."""
    rng = np.random.default_rng(T)
    rows = int(max(pos.max(), 0)) + 1
    tab = ref.rope_table(rows, rot) if rot else None
    row = (Hq + 2 * Hkv) * D + extra
    shape = (n_pages, Hkv, page)
    bufs = {n: rng.integers(0, 256, (*shape, D // 2 if len(n) == 1 else D // 32)).astype(np.uint8)
            for n in ("k", "v", "ks", "vs")}
    want = {n: b.copy() for n, b in bufs.items()}
    f = x.float().numpy()[:, :row - extra].reshape(T, Hq + 2 * Hkv, D)
    q_want = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16)
    for t in range(T):
        if seq[t] < 0 or pos[t] < 0 or seq[t] >= table.shape[0] or pos[t] // page >= table.shape[1]:
            continue
        pg, sl = int(table[seq[t], pos[t] // page]), int(pos[t] % page)
        if pg < 0 or pg >= n_pages:
            continue
        with np.errstate(over="ignore", invalid="ignore"):
            r = ref.rotate_f32(f[t:t + 1, :Hq + Hkv], tab[pos[t]][None], rot, pairs) if rot else f[t:t + 1, :Hq + Hkv]
        q_want[t] = ref.bf16(r[0, :Hq])
        for n, new in (("k", r[0, Hq:]), ("v", f[t, Hq + Hkv:])):
            want[n][pg, :, sl], want[n + "s"][pg, :, sl] = fp4_rows(new)
    d = {n: torch.from_numpy(b).to(DEV) for n, b in bufs.items()}
    c = moe.make_kv_cache(FP4, n_pages, page, Hkv, D, d["k"], d["v"], d["ks"], d["vs"])
    xd = x.to(DEV)
    q_out = torch.full((T, Hq, D), 5.0, dtype=torch.bfloat16, device=DEV) if Hq else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    at, sd, pd, td = xd.data_ptr(), i32(seq), i32(pos), i32(table)
    tabd = torch.from_numpy(tab).to(DEV) if rot else None
    moe.kv_append_rope(c, at if Hq else None, row, Hq, at + 2 * Hq * D, row, at + 2 * (Hq + Hkv) * D,
                       row, T, tabd, rows if rot else 0, rot, moe.ROPE_PAIRS if pairs else moe.ROPE_HALF,
                       sd, pd, td, table.shape[0], table.shape[1], q_out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    if Hq:
        assert torch.equal(q_out.cpu().view(torch.int16), q_want.view(torch.int16))
    got = {n: t.cpu().numpy() for n, t in d.items()}
    for n in ("ks", "vs"):
        assert np.array_equal(got[n], want[n]), n
    for n in ("k", "v"):
        none = np.repeat(want[n + "s"] == 255, 16, -1)      # (their codes say nothing)
        assert np.array_equal(got[n][~none], want[n][~none]), n


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_matches_the_rule(D, pairs):
    rng = np.random.default_rng(D + pairs)
    for T, Hq, Hkv, page, rot, extra in [(1, 1, 1, 16, D, 0), (5, 6, 2, 16, D // 2, 8), (33, 32, 8, 64, 16, 0),
                                         (7, 0, 3, 32, 0, 16), (1100, 3, 1, 128, D, 0)]:
        print(D, pairs, T, Hq, Hkv, page, rot, flush=True)
        B, cols = min(T, 9), 6
        n_pages = B * cols + 3
        table = rng.permutation(n_pages)[:B * cols].reshape(B, cols)
        flat = rng.permutation(B * cols * page)[:T]
        x = ref.bf16(rng.standard_normal((T, (Hq + 2 * Hkv) * D + extra)).astype(np.float32))
        append(x, T, Hq, Hkv, D, page, rot, pairs, flat // (cols * page), flat % (cols * page), table,
               n_pages, extra)


def test_append_at_the_edges_of_the_rule():
    """Every bf16 of a binade beside largest values whose halves are ties; zeros of both signs;
    subnormals; the largest bf16 (the scale ends at 2^125); NaN and infinities in one group of a row."""
    D, T = 64, 48
    rng = np.random.default_rng(0)
    x = np.zeros((T, 2 * D), np.float32)
    ties = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -.25, -.75, -1.25, -1.75,
                     -2.5, -3.5, -5, -6, -0.0], np.float32)
    for t in range(T):
        top = (1 + t % 16 / 16) * 2.0 ** (t // 16)             # largest: through 6 and 3 in steps
        x[t, :32] = top * np.concatenate([ties, ties[:8]]) / 6
        x[t, 32:64] = ties[t % 24]
        x[t, 64:] = (rng.standard_normal(D) * 2.0 ** (t - 24)).astype(np.float32)
    x[40, :64], x[41, :64] = -0.0, 0.0
    x[42, :64] = np.ldexp(1.0 + np.arange(64) / 64, -130)
    x[43, :64] = np.ldexp(np.arange(64.), -133)
    x[44, :64] = np.ldexp(1.9921875, 127) * np.where(np.arange(64) % 3 == 0, 1, 0.3)
    x[45, 5], x[46, 40], x[47, 70] = np.nan, np.inf, -np.inf
    append(ref.bf16(x), T, 0, 1, D, 16, 0, False, np.zeros(T, int), np.arange(T), np.array([[2, 0, 1]]), 4)


def test_append_padding_and_out_of_range():
    rng = np.random.default_rng(1)
    table = np.array([[0, 1], [2, -1], [9, 3]])
    x = ref.bf16(rng.standard_normal((4, 4 * 64)).astype(np.float32))
    append(x, 4, 2, 1, 64, 16, 64, False, np.array([-1, 0, 0, 1]), np.array([3, -5, 31, 4]), table, 4)
    append(x, 4, 2, 1, 64, 16, 0, False, np.array([3, 0, 1, 2]), np.array([0, 32, 16, 5]), table, 4,
           status=moe.MOE_STATUS_BAD_PAGE)


# ---- attention --------------------------------------------------------------------

@pytest.mark.parametrize("shape", FEW + SHAPES + TILES)
def test_matches_64_bit_attention(shape):
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, flush=True)
    rng = np.random.default_rng(B * 100 + P)
    kv, q, pre, table, n = build4(rng, B, Q, Hq, Hkv, D, page, P, own)
    pos = positions(own, P, Q)
    o, lse = call(kv, q, pos, pre, P, table, n, D ** -0.5, Q, extra=8)
    check(o, lse, q, kv, pos, pre, P, table, D ** -0.5, Q, n)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales_of_all_sizes(D):
    """Scale bytes over their whole range in V, block by block (the values' own tolerance holds for
    each output column by itself), and over a range that scores bear in K."""
    rng = np.random.default_rng(D)
    for B, Q, G in ((3, 1, 4), (3, 50, 4), (3, 180, 4)):   # few rows, more, many
        P, own = 150, [30 + Q, 64 + Q, 1 + Q]
        kv, q, pre, table, n = build4(rng, B, Q, G, 1, D, 32, P, own)
        shape = kv.t["vs"].shape
        kv.t["vs"] = torch.from_numpy((rng.integers(0, 253, shape[-1])[None] + np.zeros(shape, int)).astype(np.uint8))
        kv.t["vs"][..., 0], kv.t["vs"][..., -1] = 10, 240
        kv.t["ks"] = torch.from_numpy(rng.integers(115, 130, shape).astype(np.uint8))
        pos = positions(own, P, Q)
        o, lse = call(kv, q, pos, pre, P, table, n, 0.05, Q)
        # the tolerance of check(), and half a step of what is below the least normal: bf16's steps
        # there are 2^-133, whatever the value (an output of 7.1e-40 lies between 6.4e-40 and 7.3e-40)
        eo, el, mag, qk = ref.attention(q.double().numpy(), kv, pos, pre, P, table, 0.05, Q, n)
        d = 2 * D * 2.0 ** -23 * qk
        tol = 1.05 * 2.0 ** -8 * (mag + np.abs(eo)) + (2 * d[..., None] + 2.0 ** -16) * mag + 2.0 ** -134
        # sums are formed of weights up to 8 before they are divided: 8 x 394 keys x 6 x 2^(byte - 127)
        # is below fp32's 2^128 up to byte 240; beyond that a sum may be infinite where out is not
        fits = np.repeat(kv.t["vs"][0, 0, 0].numpy() <= 240, 32)
        assert fits.sum() >= D - 32
        assert (np.abs(o - eo) <= tol)[..., fits].all()
        assert (np.abs(lse - el) <= d + 2.0 ** -20 * (1 + np.abs(el))).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_key_gives_its_value_at_every_scale(D):
    """A row of one key has weight 1: out is V, whatever its scale byte (0 to 252)."""
    rng = np.random.default_rng(D)
    for B, P in ((1, 0), (140, 1), (520, 1)):          # few rows, more, many
        kv, q, pre, table, n = build4(rng, B, 1, 1, 1, D, 16, P, [1 - P] * B)
        pg = int(pre[0]) if P else int(table[0, 0])
        for lo in range(0, 253, D // 32):
            bytes_ = np.minimum(np.arange(lo, lo + D // 32), 252)
            kv.t["vs"][pg, 0, 0] = torch.from_numpy(bytes_.astype(np.uint8))
            o, _ = call(kv, q, np.zeros(B, int), pre, P, table, 1, 0.1, 1)
            assert np.array_equal(o, np.broadcast_to(kv.values("v")[pg, 0, 0], o.shape)), lo


def test_limits_inside_the_prefix_and_empty_rows():
    rng = np.random.default_rng(5)
    B, Q, Hq, Hkv, D, page, P = 6, 2, 4, 2, 64, 16, 70
    kv, q, pre, table, n = build4(rng, B, Q, Hq, Hkv, D, page, P, [50] * B)
    pos = np.array([-1, -1, 0, 5, 68, 69, 70, 71, -1, 119, 31, 32])
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    check(o, lse, q, kv, pos, pre, P, table, 0.125, Q, n)
    o, lse = call(kv, q, np.full(12, -1), pre, P, table, n, 0.125, Q)
    assert (o == 0).all() and (lse == -np.inf).all()
    for shape in MANY + TILES:
        B, Q, Hq, Hkv, D, page, P, own = shape
        kv, q, pre, table, n = build4(rng, B, Q, Hq, Hkv, D, page, P, own)
        pos = np.minimum(rng.integers(-30, n, B * Q), np.repeat([P + m for m in own], Q) - 1)
        o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q)
        check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)


@pytest.mark.parametrize("byte", [253, 254, 255])
@pytest.mark.parametrize("shape", MANY + TILES[:3] + [FEW[5], FEW[6], FEW[8]])
def test_what_a_row_does_not_see_does_not_enter(shape, byte):
    """NaN blocks in the free part of pages, and in one block of V at the keys of the sequences' last
    rows: those rows alone turn NaN, in that block's columns alone."""
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, byte, flush=True)
    rng = np.random.default_rng(6)
    own = [max(m, 2) for m in own]
    kv, q, pre, table, n = build4(rng, B, Q, Hq, Hkv, D, page, P, own)
    pos = positions(own, P, Q)
    pos[0] = P // 2
    want = ref.attention(q.double().numpy(), kv, pos, pre, P, table, 0.125, Q, n)
    used = {(int(pre[j // page]), j % page) for j in range(P)} | \
        {(int(table[b, j // page]), j % page) for b in range(B) for j in range(P, P + own[b])}
    for pg in range(kv.t["k"].shape[0]):
        for s in range(page):
            if (pg, s) not in used:
                kv.t["ks"][pg, :, s] = kv.t["vs"][pg, :, s] = byte
    dirty = np.zeros(B * Q, bool)
    for b in range(B):
        j = P + own[b] - 1
        kv.t["vs"][int(table[b, j // page]), :, j % page, 1] = byte
        dirty |= (np.arange(B * Q) // Q == b) & (pos >= j)
    o, lse = call(kv, q, pos, pre, P, table, n, 0.125, Q)
    assert dirty.any() and not dirty.all()
    assert np.isnan(o[dirty][..., 32:64]).all()
    compare(o, lse, q, want, ~dirty)
    others = np.r_[0:32, 64:D]
    tol = 1.05 * 2.0 ** -8 * (want[2] + np.abs(want[0])) + 2.0 ** -12 * want[2]
    assert (np.abs(o - want[0]) <= tol)[dirty][..., others].all()


def test_a_nan_key_that_a_row_sees_gives_nan():
    rng = np.random.default_rng(7)
    kv, q, pre, table, n = build4(rng, 2, 1, 4, 2, 128, 16, 40, [9, 9])
    kv.t["ks"][int(table[1, 44 // 16]), 1, 44 % 16, 2] = 255
    pos = positions([9, 9], 40, 1)
    o, lse = call(kv, q, pos, pre, 40, table, n, 0.1, 1)
    assert np.isfinite(o[0]).all() and np.isfinite(o[1, :2]).all()
    assert np.isnan(o[1, 2:]).all() and np.isnan(lse[1, 2:]).all()


def test_bad_pages():
    rng = np.random.default_rng(9)
    for shape in MANY[:2] + TILES[:2] + [FEW[4]]:
        B, Q, Hq, Hkv, D, page, P, own = shape
        kv, q, pre, table, n = build4(rng, B, Q, Hq, Hkv, D, page, P, own)
        pos = positions(own, P, Q)
        pre, table = pre.copy(), table.copy()
        pre[len(pre) // 2] = 10 ** 6
        b = int(np.argmax(own))
        table[b, (P + own[b] - 1) // page] = -5
        o, lse = call(kv, q, pos, pre, P, table, n, 0.1, Q, expect_status=moe.MOE_STATUS_BAD_PAGE)
        check(o, lse, q, kv, pos, pre, P, table, 0.1, Q, n)


def test_cache_past_4_gib():
    """Codes in the last pages of over 4 GiB of them: appended there, and read back by attention."""
    Hkv, D, page = 8, 128, 64
    n_pages = (1 << 32) // (Hkv * D // 2 * page) + 4
    k = torch.zeros((n_pages, Hkv, page, D // 2), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    ks = torch.full((n_pages, Hkv, page, D // 32), 127, dtype=torch.uint8, device=DEV)
    vs = ks.clone()
    c = moe.make_kv_cache(FP4, n_pages, page, Hkv, D, k, v, ks, vs)
    T = 100
    x = torch.randn((T, 2 * Hkv * D), device=DEV).to(torch.bfloat16)
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device=DEV)
    seq, pos = torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    moe.kv_append_rope(c, None, 0, 0, x, 2 * Hkv * D, x.data_ptr() + 2 * Hkv * D, 2 * Hkv * D, T, None, 0, 0,
                       0, seq, pos, table, 1, 2, None, None)
    q = torch.randn((1, Hkv, D), device=DEV).to(torch.bfloat16)
    nb = moe.attn_workspace_bytes(c, 1, 1, Hkv, 0, T)
    ws, o = torch.empty(nb, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    moe.attn_shared_prefix(c, q, Hkv * D, 1, 1, Hkv, pos[-1:], None, 0, table, 2, T, 0.1, o, None, None, ws, nb)
    torch.cuda.synchronize()
    f = x.float().cpu().numpy().reshape(T, 2, Hkv, D)
    val = []
    for i in range(2):
        codes, sb = fp4_rows(f[:, i])
        cell = np.empty((T, Hkv, D))
        cell[..., 0::2], cell[..., 1::2] = ref.E2M1[codes & 15], ref.E2M1[codes >> 4]
        val.append(cell * np.repeat(np.ldexp(1.0, sb.astype(int) - 127), 32, -1))
    s = np.einsum("thd,hd->ht", val[0], q[0].double().cpu().numpy()) * 0.1
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    want, mag = np.einsum("ht,thd->hd", p, val[1]), np.einsum("ht,thd->hd", p, np.abs(val[1]))
    err = np.abs(o[0].double().cpu().numpy() - want)
    assert (err <= 1.05 * 2.0 ** -8 * (mag + np.abs(want)) + 2.0 ** -12 * mag).all()
    assert int((k != 0).any(-1).any(-1).any(-1).sum()) == 2


def test_graph_replays_of_append_and_attention():
    """A step's append and attention captured together, replayed over growing positions beside eager
    steps on caches of their own."""
    rng = np.random.default_rng(2)
    B, Hq, Hkv, D, page, P = 5, 8, 2, 128, 16, 50
    kv, q, pre, table, n = build4(rng, B, 1, Hq, Hkv, D, page, P, [40] * B)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)  # noqa: E731
    table = table.copy()
    tab_d, pre_d = i32(table), i32(pre)
    rope = torch.from_numpy(ref.rope_table(n, D)).to(DEV)
    x = torch.randn((B, (Hq + 2 * Hkv) * D), device=DEV).to(torch.bfloat16)
    pos, seq = i32([P] * B), i32(range(B))
    sides = []
    for _ in range(2):
        d = {m: t.to(DEV) for m, t in kv.t.items()}
        c = moe.make_kv_cache(FP4, d["k"].shape[0], page, Hkv, D, d["k"], d["v"], d["ks"], d["vs"])
        nb = moe.attn_workspace_bytes(c, B, 1, Hq, P, n)
        sides.append(dict(d=d, c=c, nb=nb, ws=torch.empty(nb, dtype=torch.uint8, device=DEV),
                          q=torch.empty((B, Hq, D), dtype=torch.bfloat16, device=DEV),
                          o=torch.empty((B, Hq, D), dtype=torch.bfloat16, device=DEV),
                          lse=torch.empty((B, Hq), device=DEV)))

    def step(s):
        at, row = x.data_ptr(), x.shape[1]
        moe.kv_append_rope(s["c"], at, row, Hq, at + 2 * Hq * D, row, at + 2 * (Hq + Hkv) * D, row, B, rope, n,
                           D, moe.ROPE_HALF, seq, pos, tab_d, B, table.shape[1], s["q"], None)
        moe.attn_shared_prefix(s["c"], s["q"], Hq * D, B, 1, Hq, pos, pre_d, P, tab_d, table.shape[1], n, 0.1,
                               s["o"], s["lse"], None, s["ws"], s["nb"])
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        step(sides[0])
    for i in range(4):
        x.copy_(torch.randn_like(x.float()))
        step(sides[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("q", "o", "lse"):
            assert torch.equal(sides[0][name], sides[1][name]), (i, name)
        for name in ("k", "v", "ks", "vs"):
            assert torch.equal(sides[0]["d"][name], sides[1]["d"][name]), (i, name)
        pos.add_(1)


# one kv head's rows and keys at both sides of what chooses blocks of 16 or 32 rows or key tiles in LDS
LIMITS = [
    (24, 1, 4, 1, 64, 32, 8191, [1 + i % 5 for i in range(24)]),      # 96 rows: shared keys few,
    (24, 1, 4, 1, 64, 32, 8192, [1 + i % 5 for i in range(24)]),      # or many
    (24, 1, 4, 1, 128, 32, 8191, [1 + i % 5 for i in range(24)]),
    (24, 1, 4, 1, 128, 32, 8192, [1 + i % 5 for i in range(24)]),
    (24, 1, 4, 1, 128, 32, 8192, [1365] + [9] * 23),                  # 24 x 1365 < 4 x 8192 < 24 x 1366
    (24, 1, 4, 1, 128, 32, 8192, [1366] + [9] * 23),
    (40, 2, 4, 1, 64, 64, 16384, [2 + i % 5 for i in range(40)]),     # 320 rows: blocks of 32,
    (40, 2, 4, 1, 64, 64, 16385, [2 + i % 5 for i in range(40)]),     # or key tiles
    (33, 2, 4, 1, 128, 64, 16385, [2 + i % 5 for i in range(33)]),
    (1, 80, 4, 1, 64, 64, 0, [16384]),                                # a sequence's own
    (1, 80, 4, 1, 64, 64, 0, [16385]),
    (1, 24, 4, 1, 128, 16, 0, [8191]),
    (1, 24, 4, 1, 128, 16, 0, [8192]),
    (1, 16, 8, 1, 128, 64, 2000, [9000]),                             # its own by 32 rows behind few shared
    (1, 16, 8, 1, 64, 64, 2000, [8191]),
    (1, 16, 8, 1, 64, 64, 2000, [8192]),
    (1, 17, 4, 1, 128, 64, 10000, [40010]),                           # behind many, four times as many own
]


@pytest.mark.parametrize("shape", LIMITS)
def test_both_sides_of_what_chooses_the_blocks(shape):
    B, Q, Hq, Hkv, D, page, P, own = shape
    print(shape, flush=True)
    rng = np.random.default_rng(B * 100 + P)
    kv, q, pre, table, n = build4(rng, B, Q, Hq, Hkv, D, page, P, own)
    pos = positions(own, P, Q)
    o, lse = call(kv, q, pos, pre, P, table, n, D ** -0.5, Q)
    check(o, lse, q, kv, pos, pre, P, table, D ** -0.5, Q, n)
