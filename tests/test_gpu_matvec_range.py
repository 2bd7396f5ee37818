"""The 4-bit matrix-vector product at the ends of f32's range, with the bound of
tests/test_gpu_matvec.py. Every sum of terms' magnitudes is below f32's largest number, so no
order of adding them up has an excuse to overflow."""

import numpy as np
import pytest

import expert_ffn_decode_gb300 as ffn
from expert_ffn_decode_gb300 import synth
from oracle import ops_oracle as oo
from tests.test_gpu_matvec import PL, Q4K, Q40, Q41, call, check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32_MAX = 3.4028235e38


def small_weights(rng, qtype, rows, cols, size, group=64, mins=True):
    """Weights of about `size` a nibble step, so that vectors near f32's largest number have products in range."""
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    if qtype == PL:
        nib = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
        s = (size * rng.uniform(0.5, 1, (rows, cols // group))).astype(np.float16)
        m = (-8 * size * rng.uniform(0.5, 1, s.shape)).astype(np.float16) if mins else None
        return (dev(nib), dev(s), None if m is None else dev(m)), oo.planes_values(nib, s, m, group)
    n = rows * cols // synth.BLOCK_VALUES[qtype]
    b = synth.any_blocks(rng, qtype, n).reshape(n, -1)
    f16 = lambda x: np.ascontiguousarray(x.astype(np.float16)).view(np.uint8).reshape(n, 2)
    scale = size / 32 if qtype == Q4K else size  # (Q4_K: times a 6-bit scale)
    b[:, 0:2] = f16(scale * rng.uniform(0.5, 1, n))
    if qtype != Q40:
        b[:, 2:4] = f16((1 if qtype == Q4K else -8) * scale * rng.uniform(0.5, 1, n))
    b = b.reshape(rows, -1)
    return (dev(b), None, None), oo.block_values(b, cols, qtype)


CASES = [(Q40, 512, True), (Q40, 480, True), (Q41, 512, True), (Q4K, 512, True), (PL, 512, True), (PL, 512, False)]


@pytest.mark.parametrize("x_type", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 5, 9])
@pytest.mark.parametrize("qtype,cols,mins", CASES)
def test_large_vectors_of_one_sign(qtype, cols, mins, T, x_type):
    """x between 1e37 and 2e37, all of one sign: sums of x over a block pass f32's largest number
    and so do sums of q x, but not y or any sum of the terms."""
    rng = np.random.default_rng(41)
    rows = 40
    wt, val = small_weights(rng, qtype, rows, cols, 6e-4, mins=mins)
    x = rng.uniform(1e37, 2e37, (T, cols)).astype(np.float32)
    x[T - 1] *= -1
    x = torch.from_numpy(x).cuda().to(torch.float32 if x_type == "f32" else torch.bfloat16)
    ref, a = oo.matvec(*val, x.double().cpu().numpy())
    assert a.max() < F32_MAX
    y = call(wt, x, rows, cols, qtype, 64 if qtype == PL else 0)
    check(y, ref, a, 2.0 ** -24, cols)


@pytest.mark.parametrize("T", [1, 2, 5, 9])
@pytest.mark.parametrize("qtype,cols,mins", CASES)
def test_tiny_vectors(qtype, cols, mins, T):
    """x near f32's smallest normal number: results keep f32's bits down to its smallest steps."""
    rng = np.random.default_rng(42)
    rows = 40
    wt, val = small_weights(rng, qtype, rows, cols, 1.0, mins=mins)
    x = (rng.standard_normal((T, cols)) * 2.0 ** -122).astype(np.float32)
    ref, a = oo.matvec(*val, x)
    y = call(wt, torch.from_numpy(x).cuda(), rows, cols, qtype, 64 if qtype == PL else 0)
    # each of the bound's roundings may also be one of f32's smallest steps, 2^-149, off by half
    y = y.double().cpu().numpy()
    assert np.all(np.abs(y - ref) <= 2.0 ** -24 * np.abs(ref) + (64 + cols / 32) * (2.0 ** -24 * a + 2.0 ** -150))
