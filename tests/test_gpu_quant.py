"""Products of a few rows with a 4-bit matrix (include/moe_quant.h) against
float64, through the C ABI.

The kernel sums products x (16 + c) exactly formed in FP32, with 24 times the
group's sum of x taken off in the same accumulators; so with |16 + c| + 24 <=
55 the error of one result is at most 2^-24 L S before its final rounding,
S = 55 sum_k |x_k| scale_k and L the longest chain of FP32 additions: twice a
group (the sum of x, then the products), the groups of one wavefront's
sixteenth of the depth, and 20 for the sum over wavefronts and the scaling.
The final rounding adds half a unit in the last place.
"""
import numpy as np
import pytest

from oracle import moe_oracle as O
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _lib():
    from compressed_expert_ffn_amd import _lib as L
    return L


def torch_dtype(dt):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[dt]


def make(n_in, n_out, group, seed=0):
    rng = np.random.default_rng(seed)
    q = rng.integers(-8, 8, (n_in, n_out)).astype(np.int8)
    scale = (rng.random((-(-n_in // group), n_out)) * 0.2 + 0.01).astype(np.float16)
    return q, scale


def rows(T, n, dt, seed=1):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, n), generator=g).to(torch_dtype(dt))


def weights64(q, scale, group):
    return q.astype(np.float64) * np.repeat(scale.astype(np.float64), group, axis=0)[:q.shape[0]]


def check(y, x, q, scale, group, dt):
    import torch
    x = x.cpu().double().numpy()
    W = weights64(q, scale, group)
    ref = x @ W
    step = torch.finfo(torch_dtype(dt)).eps / 2
    L = 2 * group + -(-q.shape[0] // (16 * group)) + 20
    S = 55 * (np.abs(x) @ np.repeat(scale.astype(np.float64), group, axis=0)[:q.shape[0]])
    tiny = 2.0 ** -25 if dt == "f16" else 2.0 ** -134  # half the smallest number
    acc = 2.0 ** -24 * L * S
    bar = step * (np.abs(ref) + acc) + acc + tiny
    d = np.abs(y.cpu().double().numpy() - ref)
    assert (d <= bar).all(), float((d / bar).max())
    rel = np.linalg.norm(y.cpu().double().numpy() - ref) / max(np.linalg.norm(ref), 1e-300)
    # the whole result is rounded once: within half a step of it in norm, and
    # a twentieth of one for the sums
    assert rel <= 1.05 * step, rel
    return rel


# depths and widths at the edges of groups, 32-row steps, units (128, 64 or 32
# rows) and tiles (16, 32 or 64 columns: widths from 8161 and 16321 on)
SIZES = [
    (1, 1, 1, 32), (1, 8, 16, 32), (2, 31, 15, 32), (3, 32, 17, 64), (15, 33, 63, 32), (16, 64, 64, 128),
    (17, 127, 48, 64), (31, 128, 33, 128), (32, 129, 100, 32), (33, 136, 40, 128), (65, 255, 18, 64),
    (4, 1000, 77, 128), (1, 4096, 128, 32), (8, 2040, 96, 64), (1, 96, 8161, 32), (17, 200, 8170, 128),
    (2, 72, 8200, 64), (1, 160, 16321, 128), (32, 96, 16384, 32), (5, 65, 16400, 64),
]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,n_in,n_out,group", SIZES)
def test_matvec_matches_float64(T, n_in, n_out, group, dt):
    L = _lib()
    say(f"[quant] T={T} {n_in}x{n_out} group {group} {dt}")
    q, scale = make(n_in, n_out, group)
    lin = L.QuantLinear(n_in, n_out, group, dt, q=q, scale=scale)
    x = rows(T, n_in, dt)
    y = lin.matvec(x.cuda())
    rel = check(y, x, q, scale, group, dt)
    q2, s2 = lin.read()
    assert np.array_equal(q2, q) and np.array_equal(s2, scale)
    assert lin.stored_bytes() >= n_in * n_out // 2
    say(f"[quant] rel {rel:.2e}")
    lin.close()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("device", [False, True])
def test_values_are_quantised_by_the_residual_rule(dt, src, device):
    """Codes and scales bit for bit those of the layer's INT4 rule; columns of
    zeros, of one spike and of values below the smallest fp16 scale among them."""
    import torch
    L = _lib()
    n_in, n_out, group = 192, 70, 32
    rng = np.random.default_rng(3)
    v = rng.standard_normal((n_in, n_out)).astype(np.float32)
    v[:, 0] = 0
    v[:, 1] = 0
    v[5, 1] = -3.0
    v[:, 2] *= 1e-9
    v[:, 3] = np.float32(7.0) * 0.5  # exact codes 7
    v[::2, 4] = 2.5 * 0.25
    v[0, 4] = 7 * 0.25  # ties at half codes
    t = torch.from_numpy(v)
    if src != "f32":
        t = t.to(torch_dtype(src))
    ref_q, ref_s = O.quantize_int4_g32(t.float().numpy())
    arg = t.cuda() if device else t
    lin = L.QuantLinear(n_in, n_out, group, dt, values=arg)
    q, s = lin.read()
    assert np.array_equal(s.view(np.uint16), ref_s.view(np.uint16))
    assert np.array_equal(q, ref_q)
    x = rows(3, n_in, dt)
    check(lin.matvec(x.cuda()), x, q, s, group, dt)
    lin.close()


@pytest.mark.parametrize("group", [64, 128])
def test_wider_groups_share_one_scale(group):
    import torch
    L = _lib()
    n_in, n_out = 300, 20  # the last group is short
    v = np.random.default_rng(4).standard_normal((n_in, n_out)).astype(np.float32)
    lin = L.QuantLinear(n_in, n_out, group, "f16", values=torch.from_numpy(v).cuda())
    q, s = lin.read()
    for b in range(s.shape[0]):
        blk = v[b * group:(b + 1) * group]
        want = (np.abs(blk).max(axis=0) / np.float32(7.0)).astype(np.float16)
        assert np.array_equal(want.view(np.uint16), s[b].view(np.uint16))
        code = np.clip(np.rint(blk / want.astype(np.float32)), -8, 7).astype(np.int8)
        assert np.array_equal(code, q[b * group:(b + 1) * group])
    lin.close()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n_in,offset,pitch", [(128, 0, 136), (128, 1, 131), (130, 3, 130), (127, 2, 160), (128, 8, 129)])
def test_strided_and_unaligned_rows(n_in, offset, pitch, dt):
    """Rows at any pitch and alignment of their type; what lies between and
    behind the rows of Y stays as it was."""
    import torch
    L = _lib()
    T, n_out, group = 5, 50, 32
    q, scale = make(n_in, n_out, group, 5)
    lin = L.QuantLinear(n_in, n_out, group, dt, q=torch.from_numpy(q).cuda(), scale=torch.from_numpy(scale).cuda())
    x = rows(T, n_in, dt, 6)
    buf = torch.full((offset + T * pitch + 64,), float("nan"), dtype=x.dtype, device="cuda")
    xs = buf[offset:offset + T * pitch].view(T, pitch)[:, :n_in]
    xs.copy_(x)
    ybuf = torch.full((T + 2, n_out + 7), 42.0, dtype=x.dtype, device="cuda")
    y = lin.matvec(xs, ybuf[1:1 + T, 3:3 + n_out])
    check(y, x, q, scale, group, dt)
    out = ybuf.clone()
    out[1:1 + T, 3:3 + n_out] = 42.0
    assert (out == 42.0).all()
    # the same rows, packed and aligned: the same sums
    assert torch.equal(lin.matvec(x.cuda()), y)
    lin.close()


def test_rows_do_not_meet():
    """A row's result does not depend on its batch, and a row with a NaN or an
    infinity spoils only itself."""
    import torch
    L = _lib()
    n_in, n_out, group = 256, 80, 64
    q, scale = make(n_in, n_out, group, 7)
    for dt in ("f16", "bf16"):
        lin = L.QuantLinear(n_in, n_out, group, dt, q=q, scale=scale)
        x = rows(32, n_in, dt, 8).cuda()
        y = lin.matvec(x)
        for T in (1, 7, 16, 17):
            assert torch.equal(lin.matvec(x[:T]), y[:T])
        bad = x.clone()
        bad[3, 200] = float("nan")
        bad[20, 0] = float("inf")
        yb = lin.matvec(bad)
        assert yb[3].isnan().all() and yb[20].isnan().all()
        keep = [t for t in range(32) if t not in (3, 20)]
        assert torch.equal(yb[keep], y[keep])
        big = torch.full_like(x[:2], torch.finfo(x.dtype).max / 4)
        big[1] = torch.finfo(x.dtype).tiny
        ref = big.double().cpu().numpy() @ weights64(q, scale, group)
        got = lin.matvec(big).double().cpu().numpy()
        over = np.abs(ref) > 2 * torch.finfo(x.dtype).max
        assert np.isinf(got[over]).all() and (np.sign(got[over]) == np.sign(ref[over])).all()
        assert np.isfinite(got[1]).all()
        lin.close()


def test_no_rows_and_refusals():
    import torch
    L = _lib()
    q, scale = make(64, 48, 32)
    lin = L.QuantLinear(64, 48, 32, "f16", q=q, scale=scale)
    x = rows(4, 64, "f16").cuda()
    assert lin.matvec(x[:0]).shape == (0, 48)
    with pytest.raises(ValueError, match="rows overlap"):
        lin.matvec(torch.as_strided(x, (3, 64), (32, 1)))
    with pytest.raises(ValueError, match="consecutive"):
        lin.matvec(torch.as_strided(x, (1, 64), (64, 2)))
    with pytest.raises(ValueError, match="rows, X has"):
        lin.matvec(x, torch.empty((3, 48), dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError, match="torch.float16"):
        lin.matvec(x.bfloat16())
    for args in ((x.data_ptr(), 63, 1, x.data_ptr() + 256, 48), (x.data_ptr(), 64, 1, x.data_ptr() + 256, 47),
                 (x.data_ptr(), 64, -1, x.data_ptr() + 256, 48), (None, 64, 1, x.data_ptr(), 48),
                 (x.data_ptr(), 64, 1, None, 48), (x.data_ptr(), 64, 1, x.data_ptr(), 48),
                 (x.data_ptr() + 1, 64, 1, x.data_ptr() + 256, 48)):
        assert L.lib.moe_quant_matvec(lin.h, *args, None) == L.MOE_ERR_INVALID_ARG, args
    with pytest.raises(L.MoEError, match="code outside"):
        L.QuantLinear(64, 48, 32, "f16", q=np.full((64, 48), 8, np.int8), scale=scale)
    lin.close()


def test_streams_and_graph_replays():
    """One handle on two streams at once (it holds no state), and captured: the
    replays follow the inputs and equal the eager results."""
    import torch
    L = _lib()
    n_in, n_out, group = 1024, 640, 32
    q, scale = make(n_in, n_out, group, 9)
    lin = L.QuantLinear(n_in, n_out, group, "bf16", q=q, scale=scale)
    xs = [rows(T, n_in, "bf16", 10 + T).cuda() for T in (1, 9)]
    want = [lin.matvec(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(lin.matvec(xs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in outs[i])
    X, Y = xs[1].clone(), torch.empty_like(want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lin.matvec(X, Y)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.matvec(X, Y)
    for rep in range(4):
        X.copy_(xs[1] * (rep + 1))
        Y.zero_()
        eager = lin.matvec(X.clone())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager), rep
    lin.close()


def test_weights_on_another_device_than_the_current_one_are_refused(monkeypatch):
    import torch
    from compressed_expert_ffn_amd import _lib as L
    q = torch.zeros((64, 32), dtype=torch.int8, device="cuda")
    scale = torch.ones((2, 32), dtype=torch.float16, device="cuda")
    base = torch.zeros((2, 64, 64), dtype=torch.float16, device="cuda")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        L.QuantLinear(64, 32, 32, "f16", q=q, scale=scale)
    cfg = L.make_config(4, 64, 64, 2, 1, 1, 1, 0, "gelu_tanh", "f16", "f16", "none")
    with pytest.raises(ValueError, match="current"):
        L.Layer(cfg, dict(W_grp=torch.zeros((64, 2), device="cuda"), base=[base, base]), on_device=True)
