"""w4_linear against the dequantised product in 64 bits.

Tolerance: products of codes and bf16 activations are exact in fp32; an fp32
sum of K terms in any order is off by at most about sqrt(K) roundings of its
partial sums, 2^-24 each (2^-23 allowed for the matrix cores' own adds): every
output within 8 sqrt(K) 2^-23 sum |x| |w| of the exact value (for INT4 the sum
of |x| scale (code + zero), since codes and zero points are summed apart), plus
half a unit of bf16 for bf16 outputs; f32 outputs also within 1e-6 in norm."""
import numpy as np
import pytest
import torch

import ops_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


def make(rng, fmt, N, K, group, zeros=False):
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    n_g = -(-K // group)
    if fmt == "fp4":
        return q, rng.integers(119, 124, (N, n_g), dtype=np.uint8), None
    s = torch.from_numpy(rng.uniform(0.002, 0.02, (N, n_g)).astype(np.float32)).to(torch.bfloat16)
    return q, s, rng.integers(0, 16, (N, n_g), dtype=np.uint8) if zeros else None


def call(fmt, N, K, group, q, scale, zero, x, x_stride=None, y_stride=None, f32=True, stream=None):
    f = moe.MOE_W_FP4_E2M1_UE8M0_K32 if fmt == "fp4" else moe.MOE_W_INT4_BF16_GROUP
    dev = [torch.as_tensor(a).to(DEV) if a is not None else None for a in (q, scale, zero)]
    w = moe.make_w4(f, N, K, group, *dev)
    T = x.shape[0]
    xs, ys = x_stride or K, y_stride or N
    xd = torch.full((T, xs), float("nan"), dtype=torch.bfloat16)
    xd[:, :K] = x
    xd = xd.to(DEV)
    y = torch.full((T, ys), -7.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    moe.w4_linear(w, xd, xs, T, y, ys, moe.MOE_DT_F32 if f32 else moe.MOE_DT_BF16, stream)
    torch.cuda.synchronize()
    assert (y[:, N:] == -7.0).all()
    return y[:, :N].double().cpu().numpy()


def check(y, x, w, mag, K, f32):
    xd = x.double().numpy()
    exact, bound = xd @ w.T, np.abs(xd) @ mag.T
    tol = 8 * np.sqrt(K) * 2.0 ** -23 * bound
    if not f32:
        tol = tol + 2.0 ** -8 * np.abs(exact)   # bf16: 8 significant bits, half a unit 2^-8
    assert (np.abs(y - exact) <= tol).all(), np.max(np.abs(y - exact) / (tol + 1e-300))
    if f32 and np.linalg.norm(exact):
        assert np.linalg.norm(y - exact) <= 1e-6 * np.linalg.norm(exact)


@pytest.mark.parametrize("fmt,group,zeros", [("fp4", 32, False), ("int4", 32, True),
                                             ("int4", 64, False), ("int4", 128, True)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 16, 17, 33, 64, 65])
def test_matches_the_dequantised_product(fmt, group, zeros, T):
    rng = np.random.default_rng(T + group)
    for N, K, pad, f32 in [(1, 32, 0, True), (17, 96, 8, False), (100, 288, 0, True),
                           (257, 1056, 64, True), (48, 4096, 0, False), (33, 8224, 8, True)]:
        print(fmt, group, T, N, K, flush=True)
        q, s, z = make(rng, fmt, N, K, group, zeros)
        x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
        y = call(fmt, N, K, group, q, s, z, x, K + pad, N + pad // 8, f32)
        check(y, x, *ref.w4_dequant(fmt, q, s, z, group), K, f32)


@pytest.mark.parametrize("fmt", ["fp4", "int4"])
@pytest.mark.parametrize("T", [1, 6])
def test_many_rows(fmt, T):
    rng = np.random.default_rng(5)
    N, K = 20011, 512
    q, s, z = make(rng, fmt, N, K, 32, True)
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    check(call(fmt, N, K, 32, q, s, z, x), x, *ref.w4_dequant(fmt, q, s, z, 32), K, True)


@pytest.mark.parametrize("T", [1, 2, 7, 20])
def test_every_code_and_scale(T):
    """One weight per output against one activation of 1: the dequantised value
    itself, over every code and scales from 2^-100 to 2^100; scale 255 is NaN."""
    rng = np.random.default_rng(0)
    bytes_ = [27, 100, 126, 127, 128, 160, 227]
    rows = [(c, b) for c in range(16) for b in bytes_]
    q = np.zeros((len(rows), 32), np.uint8)
    s = np.full((len(rows), 2), 127, np.uint8)
    for i, (c, b) in enumerate(rows):
        j = int(rng.integers(0, 64))
        q[i, j // 2] = c << (4 * (j & 1))
        s[i, j // 32] = b
    x = torch.ones((T, 64), dtype=torch.bfloat16)
    w, _ = ref.w4_dequant("fp4", q, s, None, 32)
    y = call("fp4", len(rows), 64, 32, q, s, None, x)
    assert np.array_equal(y, np.broadcast_to(w.sum(1), y.shape))
    s[3, 1] = 255
    y = call("fp4", len(rows), 64, 32, q, s, None, x)
    assert np.isnan(y[:, 3]).all() and np.isfinite(np.delete(y, 3, 1)).all()


@pytest.mark.parametrize("fmt", ["fp4", "int4"])
@pytest.mark.parametrize("T", [2, 5, 40])
def test_nan_and_inf_stay_in_their_token(fmt, T):
    rng = np.random.default_rng(3)
    N, K = 40, 160
    q, s, z = make(rng, fmt, N, K, 32)
    q |= 0x11          # no code is 0
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    clean = call(fmt, N, K, 32, q, s, z, x)
    x[1, 7] = float("nan")
    if T > 2:
        x[T - 1, K - 1] = float("inf")
    y = call(fmt, N, K, 32, q, s, z, x)
    bad = [1] + ([T - 1] if T > 2 else [])
    assert not np.isfinite(y[bad]).any()
    assert np.array_equal(np.delete(y, bad, 0), np.delete(clean, bad, 0))


def test_another_stream_and_graph():
    rng = np.random.default_rng(9)
    N, K, T = 64, 256, 3
    q, s, z = make(rng, "fp4", N, K, 32)
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    st = torch.cuda.Stream()
    assert np.array_equal(call("fp4", N, K, 32, q, s, z, x),
                          call("fp4", N, K, 32, q, s, z, x, stream=st))


def test_empty_batch_leaves_the_output():
    w = moe.make_w4(1, 16, 32, 32, torch.zeros(16, 16, dtype=torch.uint8, device=DEV),
                    torch.zeros(16, 1, dtype=torch.uint8, device=DEV))
    y = torch.full((4, 16), 3.0, device=DEV)
    moe.w4_linear(w, torch.zeros(4, 32, dtype=torch.bfloat16, device=DEV), 32, 0, y, 16,
                  moe.MOE_DT_F32)
    torch.cuda.synchronize()
    assert (y == 3.0).all()
