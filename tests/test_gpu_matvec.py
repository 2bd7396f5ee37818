"""The 4-bit matrix-vector product on the GPU against the float64 oracle.

Tolerance, element by element: y is rounded once (half a step of its type, relative to y),
and before that every operation is an f32 rounding or finer of terms whose magnitudes sum to
`a` (the oracle's second result). At most 32 roundings inside a block, one for each block and
32 for joining partial sums and splitting x act on a term: (64 + cols / 32) 2^-24 a."""

import numpy as np
import pytest

import expert_ffn_decode_gb300 as ffn
from expert_ffn_decode_gb300 import synth
from oracle import ops_oracle as oo

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": (ffn.MOE_F32, torch.float32, 2.0 ** -24), "f16": (ffn.MOE_F16, torch.float16, 2.0 ** -11),
         "bf16": (ffn.MOE_BF16, torch.bfloat16, 2.0 ** -8)}
Q40, Q41, Q4K, PL = ffn.MOE_Q4_0, ffn.MOE_Q4_1, ffn.MOE_Q4_K, ffn.MOE_Q4_PLANES


def make_weights(rng, qtype, rows, cols, group=0, mins=False):
    """(device tensors w, scales, mins; the oracle's (q, scale, offset))."""
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    if qtype == PL:
        nib = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
        s = rng.uniform(0.005, 0.02, (rows, cols // group)).astype(np.float16)
        m = rng.uniform(-0.1, 0.0, s.shape).astype(np.float16) if mins else None
        return (dev(nib), dev(s), None if m is None else dev(m)), oo.planes_values(nib, s, m, group)
    b = synth.any_blocks(rng, qtype, rows * cols // synth.BLOCK_VALUES[qtype]).reshape(rows, -1)
    return (dev(b), None, None), oo.block_values(b, cols, qtype)


def check(y, ref, a, half_step, cols, label=""):
    y = y.double().cpu().numpy()
    tol = half_step * np.abs(ref) + (64 + cols / 32) * 2.0 ** -24 * a
    bad = np.abs(y - ref) > tol
    assert not bad.any(), (label, int(bad.sum()), float((np.abs(y - ref) / tol).max()))


def call(wt, x, rows, cols, qtype, group=0, yt="f32", bias=None, y=None, flags=0, stream=None, **strides):
    xt = next(v[0] for v in TYPES.values() if v[1] == x.dtype)
    cfg = ffn.make_matvec_cfg(rows, cols, x.shape[0], qtype=qtype, group=group, x_type=xt, y_type=TYPES[yt][0],
                              flags=flags, **strides)
    if y is None:
        y = torch.full((x.shape[0], rows), float("nan"), dtype=TYPES[yt][1], device="cuda")
    ffn.check(ffn.moe_q4_matvec(x, *wt, bias, cfg, y, stream or torch.cuda.current_stream()))
    return y


SHAPES = [
    # qtype, group, mins, rows, cols, vectors, x, y
    (Q41, 0, False, 1, 32, 1, "f32", "f32"), (Q40, 0, False, 5, 96, 1, "bf16", "f32"),
    (Q40, 0, False, 16, 160, 2, "f32", "bf16"), (Q41, 0, False, 17, 128, 3, "f16", "f16"),
    (Q40, 0, False, 33, 2080, 1, "f32", "f32"), (Q41, 0, False, 100, 2048, 4, "f32", "f32"),
    (Q41, 0, False, 48, 2560, 5, "bf16", "bf16"), (Q4K, 0, False, 3, 256, 1, "f32", "f32"),
    (Q4K, 0, False, 31, 2560, 1, "bf16", "f32"), (Q4K, 0, False, 64, 512, 2, "f32", "f16"),
    (Q4K, 0, False, 65, 1280, 7, "f16", "f32"), (Q4K, 0, False, 16, 4864, 8, "f32", "f32"),
    (PL, 32, False, 7, 32, 1, "f32", "f32"), (PL, 32, True, 20, 1056, 1, "f32", "f32"),
    (PL, 64, True, 37, 2112, 5, "f16", "f16"), (PL, 128, False, 16, 128, 1, "bf16", "bf16"),
    (PL, 128, True, 50, 6784, 3, "f32", "f32"), (PL, 64, False, 129, 64, 9, "f32", "f32"),
    (Q40, 0, False, 40, 8192, 8, "f32", "f32"), (Q41, 0, False, 19, 16384, 1, "f32", "f32"),
    (Q41, 0, False, 19, 16384, 6, "f32", "f32"), (Q4K, 0, False, 20, 16384, 3, "bf16", "f32"),
    (PL, 32, True, 18, 16352, 2, "f32", "f32"), (Q40, 0, False, 2500, 320, 1, "f32", "f32"),
    (Q41, 0, False, 5000, 2048, 1, "bf16", "bf16"), (Q40, 0, False, 24, 256, 17, "f32", "f32"),
    (Q4K, 0, False, 33, 256, 40, "bf16", "f32"), (Q40, 0, False, 10007, 96, 2, "f16", "f32"),
]


@pytest.mark.parametrize("qtype,group,mins,rows,cols,T,xt,yt", SHAPES)
def test_against_oracle(qtype, group, mins, rows, cols, T, xt, yt):
    rng = np.random.default_rng(rows * 7 + cols + T)
    wt, val = make_weights(rng, qtype, rows, cols, group, mins)
    x = torch.from_numpy(rng.standard_normal((T, cols)).astype(np.float32)).to(TYPES[xt][1]).cuda()
    y = call(wt, x, rows, cols, qtype, group, yt)
    ref, a = oo.matvec(*val, x.double().cpu().numpy())
    check(y, ref, a, TYPES[yt][2], cols)
    again = call(wt, x, rows, cols, qtype, group, yt)
    assert torch.equal(y, again)  # repeat calls agree bit for bit
    one = call(wt, x[T - 1:], rows, cols, qtype, group, "f32")  # a vector alone, in another call form
    check(one, ref[T - 1:], a[T - 1:], TYPES["f32"][2], cols)


@pytest.mark.parametrize("T", [1, 3, 11])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_strides_bias_accumulate(T, yt):
    rng = np.random.default_rng(11)
    rows, cols = 53, 704
    wt, val = make_weights(rng, Q41, rows, cols)
    buf = torch.from_numpy(rng.standard_normal((T, cols + 40)).astype(np.float32)).cuda()
    x = buf[:, 8:8 + cols]
    bias = rng.standard_normal(rows).astype(np.float32)
    out = torch.from_numpy(rng.standard_normal((T, rows + 11))).to(TYPES[yt][1]).cuda()
    before = out.clone()
    call(wt, x, rows, cols, Q41, yt=yt, bias=torch.from_numpy(bias).cuda(), y=out, flags=ffn.MOE_ACCUMULATE,
         x_stride=cols + 40, y_stride=rows + 11)
    assert torch.equal(out[:, rows:], before[:, rows:])  # nothing is written past a vector's rows
    old = before[:, :rows].double().cpu().numpy()
    ref, a = oo.matvec(*val, x.double().cpu().numpy())
    check(out[:, :rows], ref + bias + old, a + np.abs(bias) + np.abs(old), TYPES[yt][2], cols)


@pytest.mark.parametrize("qtype,group", [(Q40, 0), (Q41, 0), (Q4K, 0), (PL, 64)])
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_extreme_magnitudes(qtype, group, scale):
    """Vectors far from 1, with a block of zeros and one value 1e6 times its neighbours."""
    rng = np.random.default_rng(5)
    rows, cols = 24, 512
    wt, val = make_weights(rng, qtype, rows, cols, group)
    x = rng.standard_normal((2, cols)).astype(np.float32)
    x[:, 64:96] = 0
    x[:, 200] *= 1e6
    x = (x * np.float32(scale)).astype(np.float32)
    for T in (1, 2):
        y = call(wt, torch.from_numpy(x[:T]).cuda(), rows, cols, qtype, group)
        ref, a = oo.matvec(*val, x[:T])
        check(y, ref, a, 2.0 ** -24, cols)


def test_zero_and_subnormal_scales():
    """Scales of zero and below the normal f16 range are exact."""
    rng = np.random.default_rng(6)
    rows, cols = 16, 256
    nib = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    s = (rng.integers(0, 900, (rows, 8)) * 2.0 ** -24).astype(np.float16)
    s[:, 3] = 0
    x = rng.standard_normal((1, cols)).astype(np.float32)
    wt = (torch.from_numpy(nib).cuda(), torch.from_numpy(s).cuda(), None)
    y = call(wt, torch.from_numpy(x).cuda(), rows, cols, PL, 32)
    ref, a = oo.matvec(*oo.planes_values(nib, s, None, 32), x)
    check(y, ref, a, 2.0 ** -24, cols)


@pytest.mark.parametrize("T", [2, 6])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_stays_in_its_vector(T, bad):
    rng = np.random.default_rng(7)
    rows, cols = 40, 320
    wt, val = make_weights(rng, Q40, rows, cols)
    x = rng.standard_normal((T, cols)).astype(np.float32)
    x[1, 77] = bad
    y = call(wt, torch.from_numpy(x).cuda(), rows, cols, Q40)
    assert not torch.isfinite(y[1]).any()
    keep = [t for t in range(T) if t != 1]
    ref, a = oo.matvec(*val, x[keep])
    check(y[keep], ref, a, 2.0 ** -24, cols)


def test_non_finite_single_vector():
    rng = np.random.default_rng(8)
    wt, _ = make_weights(rng, Q41, 20, 512)
    x = rng.standard_normal((1, 512)).astype(np.float32)
    x[0, 300] = np.nan
    assert not torch.isfinite(call(wt, torch.from_numpy(x).cuda(), 20, 512, Q41)).any()


@pytest.mark.parametrize("flags", [0, ffn.MOE_NO_PDL])
def test_chain_on_another_stream_and_in_a_graph(flags):
    """y2 = W2 (W1 x), each call reading what the one before wrote, launched eagerly on a side
    stream and replayed from a captured graph with new inputs."""
    rng = np.random.default_rng(9)
    n = 1024
    w1, v1 = make_weights(rng, Q41, n, n)
    w2, v2 = make_weights(rng, Q40, n, n)
    x = torch.empty(1, n, device="cuda")
    mid = torch.zeros(1, n, device="cuda")
    out = torch.zeros(1, n, device="cuda")

    def chain(st):
        for _ in range(4):
            call(w1, x, n, n, Q41, y=mid, flags=flags, stream=st)
            call(w2, mid, n, n, Q40, y=out, flags=flags, stream=st)

    def want(xv):
        m, _ = oo.matvec(*v1, xv)
        return oo.matvec(*v2, m)[0]

    st = torch.cuda.Stream()
    for seed in range(3):
        xv = np.random.default_rng(seed).standard_normal((1, n)).astype(np.float32)
        with torch.cuda.stream(st):
            x.copy_(torch.from_numpy(xv))
            chain(st)
        st.synchronize()
        ref = want(xv)
        assert np.linalg.norm(out.double().cpu().numpy() - ref) < 1e-5 * np.linalg.norm(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(torch.cuda.current_stream())
    for seed in (5, 6):
        xv = np.random.default_rng(seed).standard_normal((1, n)).astype(np.float32)
        x.copy_(torch.from_numpy(xv))
        g.replay()
        torch.cuda.synchronize()
        ref = want(xv)
        assert np.linalg.norm(out.double().cpu().numpy() - ref) < 1e-5 * np.linalg.norm(ref)


def test_rows_past_32_bits():
    """A matrix of more than 2^32 bytes: the last rows are read where they are."""
    cols = 16384
    rows = (1 << 32) // 10240 + 37
    w = torch.empty(rows, 10240, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(10)
    (tail, _, _), val = make_weights(rng, Q41, 64, cols)
    w.zero_()
    w[-64:] = tail
    x = rng.standard_normal((1, cols)).astype(np.float32)
    y = call((w, None, None), torch.from_numpy(x).cuda(), rows, cols, Q41)
    ref, a = oo.matvec(*val, x)
    check(y[:, -64:], ref, a, 2.0 ** -24, cols)
    assert not y[:, :-64].any()


def test_nothing_to_do():
    y = torch.full((1, 8), 3.0, device="cuda")
    cfg = ffn.make_matvec_cfg(8, 32, 0)
    ffn.check(ffn.moe_q4_matvec(None, None, None, None, None, cfg, y, torch.cuda.current_stream()))
    assert (y == 3).all()
