"""add_rmsnorm against 64 bits: the stored residual stream bit for bit, the norm of what is stored
within one rounding, the E4M3 codes within half a step."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"
# fp32 in the sum of squares: a thread adds 16 squares at most, its wave 6 times, the waves 16: under
# 64 roundings of 2^-24, halved by the root; the mean, the root, its reciprocal and two products: 5
# more.  Under 40 in all.
F32 = 40 * 2.0 ** -24


def call(x, res, w, eps, H, T, want_y=True, want_q=False, in_place=False, xs=None, rs=None, stream=None):
    """x, res: CPU tensors [T][stride]; returns res_out, y, q, scales (CPU)."""
    xd, rd = x.to(DEV), res.to(DEV) if res is not None else None
    wd = w.to(DEV) if w is not None else None
    ro = rd if in_place else torch.full_like(rd, 7.0) if rd is not None else None
    y = torch.full((T, H), 5.0, dtype=torch.bfloat16, device=DEV) if want_y else None
    q = torch.full((T, H), 0x55, dtype=torch.uint8, device=DEV) if want_q else None
    s = torch.full((T, H // 128), 3.0, device=DEV) if want_q else None
    dt = moe.MOE_DT_F32 if res is not None and res.dtype == torch.float32 else moe.MOE_DT_BF16
    moe.add_rmsnorm(xd, xs or x.shape[1], rd, dt, rs or (res.shape[1] if res is not None else 0), T, H, wd,
                    eps, ro, y, q, s, stream)
    torch.cuda.synchronize()
    return [t.cpu() if t is not None else None for t in (ro, y, q, s)]


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def check(x, res, w, eps, H, T, got):
    ro, y, q, s = got
    r = x[:, :H].float()
    if res is not None:
        r = (r + res[:, :H].float()).to(res.dtype)
        assert torch.equal(bits(ro[:, :H].contiguous()), bits(r.contiguous()))
        if ro.shape[1] > H:      # what lies between the rows stays
            assert bool((ro[:, H:] == 7.0).all()) or torch.equal(ro[:, H:], res[:, H:])
    r = r.double()
    e = r / torch.sqrt((r * r).mean(1, keepdim=True) + float(np.float32(eps)))
    if w is not None:
        e = e * w.double()
    if y is not None:
        tol = (2.0 ** -8 + 1.01 * F32) * e.abs() + 2.0 ** -133
        assert bool(((y.double() - e).abs() <= tol).all()), float((y.double() - e).abs().max())
    if q is not None:
        top = e.abs().unflatten(1, (-1, 128)).amax(2)
        sd = s.double()
        assert bool(((sd - top / 448).abs() <= (F32 + 2.0 ** -23) * top / 448 + 2.0 ** -149).all())
        v = q.view(torch.float8_e4m3fn).double() * sd.repeat_interleave(128, 1)
        # half a step: 2^-4 of the value, below the least normal (2^-6) 2^-10 of the scale
        tol = 2.0 ** -4 * 1.001 * e.abs() + 2.0 ** -10 * 1.001 * sd.repeat_interleave(128, 1)
        assert bool(((v - e).abs() <= tol).all()), float((v - e).abs().max())


def make(rng, T, H, res, pad=0, scale=1.0):
    x = torch.from_numpy(rng.standard_normal((T, H + pad)).astype(np.float32) * scale).to(torch.bfloat16)
    r = None
    if res:
        r = torch.from_numpy(4 * scale * rng.standard_normal((T, H + pad)).astype(np.float32))
        r = r.to(torch.bfloat16) if res == "bf16" else r
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(H)).astype(np.float32)).to(torch.bfloat16)
    return x, r, w


@pytest.mark.parametrize("res", ["bf16", "f32", None])
@pytest.mark.parametrize("H", [8, 128, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384])
def test_widths(H, res):
    rng = np.random.default_rng(H)
    for T in (1, 3, 17):
        print(H, res, T, flush=True)
        x, r, w = make(rng, T, H, res)
        check(x, r, w, 1e-6, H, T, call(x, r, w, 1e-6, H, T, True, H % 128 == 0))
    if H % 128 == 0:
        check(x, r, None, 1e-5, H, T, call(x, r, None, 1e-5, H, T, False, True))


@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_strides_and_in_place(res):
    rng = np.random.default_rng(1)
    T, H = 9, 384
    x, r, w = make(rng, T, H, res, pad=24)
    check(x, r, w, 1e-6, H, T, call(x, r, w, 1e-6, H, T, True, True))
    got = call(x, r, w, 1e-6, H, T, True, True, in_place=True)
    assert torch.equal(got[0][:, H:], r[:, H:])
    check(x, r, w, 1e-6, H, T, got)
    # no place for the stream: the outputs are the same
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    moe.add_rmsnorm(xd, H + 24, rd, moe.MOE_DT_BF16 if res == "bf16" else moe.MOE_DT_F32, H + 24, T, H,
                    wd, 1e-6, None, y, None, None)
    torch.cuda.synchronize()
    assert torch.equal(bits(y.cpu()), bits(got[1])) and torch.equal(rd.cpu(), r)


def test_many_rows_and_rows_behind_the_last():
    rng = np.random.default_rng(2)
    T, H = 3001, 256
    x, r, w = make(rng, T + 2, H, "bf16")
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    y = torch.full((T + 2, H), 5.0, dtype=torch.bfloat16, device=DEV)
    q = torch.full((T + 2, H), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((T + 2, H // 128), 3.0, device=DEV)
    moe.add_rmsnorm(xd, H, rd, moe.MOE_DT_BF16, H, T, H, wd, 1e-6, rd, y, q, s)
    torch.cuda.synchronize()
    check(x[:T], r[:T], w, 1e-6, H, T, (rd[:T].cpu(), y[:T].cpu(), q[:T].cpu(), s[:T].cpu()))
    assert torch.equal(rd[T:].cpu(), r[T:]) and bool((y[T:] == 5).all()) and bool((q[T:] == 0x55).all())
    assert bool((s[T:] == 3).all())


def test_zeros_small_and_large_rows():
    """A row of zeros; squares that underflow beside eps; squares past fp32's range, in one element and
    in all; eps of the least size."""
    H, T = 640, 6
    x = torch.zeros((T, H), dtype=torch.bfloat16)
    x[1] = 2.0 ** -100
    x[2, 5] = 2.0 ** 100
    x[3] = -(2.0 ** 127)
    x[4, ::2], x[4, 1::2] = 2.0 ** 65, 2.0 ** 40
    x[5] = 2.0 ** -120
    r = torch.zeros((T, H))
    for eps in (1e-6, 2.0 ** -100):
        check(x, r, None, eps, H, T, call(x, r, None, eps, H, T, True, True))


def test_nan_and_infinity_follow_the_formula():
    """mean = NaN or inf: a row with a NaN is NaN; one with an infinity is 0 with NaN in its place (0
    times inf).  In q a NaN keeps its place; the other rows are as they are alone."""
    H, T = 256, 4
    rng = np.random.default_rng(3)
    x, r, w = make(rng, T, H, "bf16")
    clean = call(x, r, w, 1e-6, H, T, True, True)
    x[1, 7], x[2, 200] = float("nan"), float("inf")
    ro, y, q, s = call(x, r, w, 1e-6, H, T, True, True)
    for t in (0, 3):
        for a, b in zip((ro, y, q, s), clean):
            assert torch.equal(a[t], b[t])
    v = q.view(torch.float8_e4m3fn).float()
    assert bool(y[1].isnan().all()) and bool(v[1].isnan().all())
    nan = torch.zeros(H, dtype=torch.bool)
    nan[200] = True
    assert torch.equal(y[2].isnan(), nan) and bool((y[2][~nan] == 0).all())
    assert torch.equal(v[2].isnan(), nan) and bool((v[2][~nan] == 0).all())


def test_q_equals_act_quant_where_y_is_a_bf16():
    """Rows whose norm is exact in bf16 (a constant row of a power of two: y = w, the root of 1 being
    1): the codes are act_quant_fp8's of y."""
    H, T = 512, 5
    x = torch.ones((T, H), dtype=torch.bfloat16) * torch.tensor([1., 2., 4., 8., 0.5])[:, None]
    x = x.to(torch.bfloat16)
    rng = np.random.default_rng(4)
    w = torch.from_numpy(rng.standard_normal(H).astype(np.float32)).to(torch.bfloat16)
    ro, y, q, s = call(x, None, w, 2.0 ** -100, H, T, True, True)
    assert torch.equal(bits(y), bits(w.expand(T, H).contiguous()))
    q2 = torch.empty((T, H), dtype=torch.uint8, device=DEV)
    s2 = torch.empty((T, H // 128), device=DEV)
    moe.act_quant_fp8(y.to(DEV), moe.MOE_DT_BF16, T, H, q2, s2)
    torch.cuda.synchronize()
    assert torch.equal(q, q2.cpu()) and torch.equal(s, s2.cpu())


def test_other_stream_and_captured():
    rng = np.random.default_rng(5)
    T, H = 33, 1152
    x, r, w = make(rng, T, H, "bf16")
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    ro, y = torch.empty_like(rd), torch.empty_like(xd)
    q, s = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((T, H // 128), device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def go():
        moe.add_rmsnorm(xd, H, rd, moe.MOE_DT_BF16, H, T, H, wd, 1e-6, ro, y, q, s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        go()
    for i in range(3):
        x, r, w = make(rng, T, H, "bf16")
        xd.copy_(x), rd.copy_(r), wd.copy_(w)
        for t in (ro, y, q, s):
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(x, r, w, 1e-6, H, T, [t.cpu() for t in (ro, y, q, s)])


@pytest.mark.parametrize("res", ["bf16", "f32", None])
def test_thousands_of_rows_of_up_to_4096_columns(res):
    """The blocks of 256 threads with two chunks each."""
    rng = np.random.default_rng(6)
    for T, H in ((2049, 2176), (2100, 4096)):
        print(T, H, res, flush=True)
        x, r, w = make(rng, T, H, res)
        check(x, r, w, 1e-6, H, T, call(x, r, w, 1e-6, H, T, True, True))
