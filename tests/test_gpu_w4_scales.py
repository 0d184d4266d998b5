"""w4_linear with FP4 scale bytes at both ends of their range: the same values from the
one-token kernel and from the matrix cores, exact (one weight an output, powers of two)."""
import numpy as np
import pytest
import torch

import ops_ref as ref
from test_gpu_w4_linear import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 3, 20, 40])
@pytest.mark.parametrize("x0,bytes_", [(2.0 ** -60, (250, 251, 252, 253, 254)),
                                       (1.0, (253, 252, 1, 0)), (2.0 ** 60, (0, 1, 2, 3, 4))])
def test_first_and_last_scales(T, x0, bytes_):
    """One weight of every code and scale an output, against an activation that brings the
    value back to the middle of fp32's range (or not: then a result below fp32's normal
    numbers may be 0)."""
    rng = np.random.default_rng(T)
    for K in (64, 512, 2048, 4096, 4128):
        print(T, K, x0, flush=True)
        rows = [(c, b) for c in range(16) for b in bytes_]
        q = np.zeros((len(rows), K // 2), np.uint8)
        s = np.full((len(rows), K // 32), 127, np.uint8)
        for i, (c, b) in enumerate(rows):
            j = int(rng.integers(0, K))
            q[i, j // 2] = c << (4 * (j & 1))
            s[i, j // 32] = b
        x = torch.full((T, K), x0, dtype=torch.bfloat16)
        w, _ = ref.w4_dequant("fp4", q, s, None, 32)
        want = np.broadcast_to(w.sum(1) * x0, (T, len(rows)))
        fits = np.abs(want) < 2.0 ** 128
        y = call("fp4", len(rows), K, 32, q, s, None, x)
        off = np.abs(y - want) > np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -126, 0)
        off |= ~np.isfinite(y)
        assert not (off & fits).any(), [(rows[n], y[t, n]) for t, n in np.argwhere(off & fits)[:6]]
        assert (np.abs(y[~fits]) == np.inf).all()


@pytest.mark.parametrize("T", [1, 2, 3, 20, 40])
def test_large_scales_leave_other_rows_alone(T):
    """Rows with bytes of 254 and 255 beside ordinary ones, in one tile."""
    rng = np.random.default_rng(T)
    N, K = 40, 1024
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = rng.integers(119, 124, (N, K // 32), dtype=np.uint8)
    x = ref.bf16(rng.standard_normal((T, K)).astype(np.float32))
    clean = call("fp4", N, K, 32, q, s, None, x)
    x2 = x * 2.0 ** -20
    s[5, 3], s[6, 30], s[20] = 254, 255, 253
    y = call("fp4", N, K, 32, q, s, None, x2)
    keep = [n for n in range(N) if n not in (5, 6, 20)]
    assert np.array_equal(y[:, keep], clean[:, keep] * 2.0 ** -20)
    assert np.isnan(y[:, 6]).all()
    w, mag = ref.w4_dequant("fp4", q, s, None, 32)
    xd = x2.double().numpy()
    for n in (5, 20):
        tol = 8 * np.sqrt(K) * 2.0 ** -23 * (np.abs(xd) @ mag[n])
        assert (np.abs(y[:, n] - xd @ w[n]) <= tol).all()
