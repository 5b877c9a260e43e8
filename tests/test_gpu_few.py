"""The few-token forward pass (moe_forward_few) against the CPU oracle, through
the C ABI: every storage combination, token counts at the edges of its MFMA
tiles, odd group and expert counts, layers whose sizes do not divide among
wavefronts, and the routing lists.

Bars: routing exact and gate weights to 1e-6 * max(1, sqrt(d / 1024)) as for
moe_forward.  y is rounded once, at most half a step of its type (eps / 2 of
the value).  What comes before it: FP32 sums of at most a few thousand terms
(2^-24 times the root of their number times a chain of a few hundred: under
2^-15 of the result's size) and hidden sums as two 16-bit parts (2^-22 of each
for fp16, 2^-17 for bf16, times the root of f <= 2^10 in the result: under
2^-12), i.e. at most a twentieth of eps / 2 for fp16 and bf16; in norm and, for
single values, of the largest.  fp32 layers keep the library's bar of 1e-5 of
the largest value.

bf16 activations on fp16 MFMAs (an fp16 or 4-bit base) hold each hidden sum h
(and each rank sum) as one fp16 number, off by at most 2^-11 |h|, evenly
distributed: standard deviation 2^-11 / sqrt(3) |h| at most.  Those errors are
independent, so y = sum h w is off by a standard deviation of 2^-11 / sqrt(3)
sqrt(sum h^2 w^2), and with weights of one variance sqrt(sum h^2 w^2) is the
root mean square of the token's y.  Six of these, 6 / sqrt(3) 2^-11 rms =
0.43 eps / 2 rms, are not passed by any of the 10^5 values checked (chance
2e-9 each); in norm they add in squares, (2^-11 / sqrt(3))^2 against the
(eps / 2)^2 allowed: under a hundredth.
"""
import numpy as np
import pytest

from compressed_expert_ffn_amd.workloads import WORKLOADS, Workload
from oracle import moe_oracle as O
from tests.gpu_util import rel_err, route_to_host, say, x_to_device, y_to_host
from tests.layers import make_parity_layer
from tests.test_gpu_parity import check_routing

pytestmark = pytest.mark.gpu

STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _lib():
    from compressed_expert_ffn_amd import _lib as L
    return L


def workload(act, xd, bd, resid, r, gk, kg, ke, T, d, f, bias=0.5):
    return Workload(f"few_{act}_{xd}_{bd}_{resid}", 60, T=T, d=d, f=f, G=gk[0], K=gk[1], top_groups=kg,
                    top_experts=ke, r=r, act=act, x_dtype=xd, base_dtype="f32" if bd == "int4_g32" else bd,
                    resid=resid, bias_scale=bias)


def make(act, xd, bd, resid, r, gk, kg, ke, T, d, f, bias=0.5, T_max=None, device=False):
    """(workload, oracle layer, library layer, X on the device)."""
    L = _lib()
    w, inputs, layer = make_parity_layer(workload(act, xd, bd, resid, r, gk, kg, ke, T, d, f, bias))
    if bd == "int4_g32":
        layer = dict(layer, base=[np.stack([O.dequantize_int4_g32(*O.quantize_int4_g32(b)) for b in p])
                                  for p in inputs["base"]])
    cfg = L.make_config(T if T_max is None else T_max, d, f, gk[0], gk[1], kg, ke, r, act, xd, bd, resid)
    return w, layer, L.Layer(cfg, inputs, on_device=device), x_to_device(inputs["X"], xd)


def check_y(Y, ref, xd, one_part=False):
    y = y_to_host(Y)
    assert np.isfinite(y).all()
    if xd == "f32":
        e = rel_err(y, ref)
        assert e <= 1e-5, e
        return e
    e = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    assert e <= 1.05 * STEP[xd], e
    bar = STEP[xd] * (np.abs(ref) + 0.05 * np.abs(ref).max())
    if one_part:
        bar += 6 / np.sqrt(3) * 2.0 ** -11 * np.sqrt((ref ** 2).mean(axis=1, keepdims=True))
    assert (np.abs(y - ref) <= bar).all(), float((np.abs(y - ref) / bar).max())
    return e


CASES = [
    # act, x, base, residual, r, (G, K), kg, ke, T, d, f
    ("swiglu", "f16", "f16", "f16", 16, (4, 4), 1, 2, 1, 256, 512),
    ("swiglu", "f16", "f16", "int4_g32", 16, (16, 16), 2, 4, 1, 320, 192),
    ("swiglu", "f16", "f16", "int4_g32", 16, (16, 16), 2, 4, 16, 320, 192),
    ("swiglu", "f16", "f16", "int4_g32", 5, (3, 3), 2, 3, 17, 64, 64),
    ("swiglu", "f16", "f16", "none", 0, (8, 1), 2, 1, 2, 576, 448),
    ("swiglu", "f16", "f16", "none", 0, (5, 7), 5, 3, 32, 128, 192),
    ("gelu_tanh", "f16", "f16", "f16", 16, (2, 8), 1, 3, 8, 192, 320),
    ("gelu_tanh", "f16", "f16", "int4_g32", 7, (3, 5), 2, 2, 9, 256, 64),
    ("gelu_tanh", "f16", "f16", "int4_g32", 16, (1, 1), 1, 1, 3, 64, 128),
    ("swiglu", "bf16", "bf16", "int4_g32", 16, (4, 4), 1, 2, 7, 256, 512),
    ("swiglu", "bf16", "bf16", "none", 0, (8, 1), 2, 1, 31, 1024, 320),
    ("gelu_tanh", "bf16", "bf16", "int4_g32", 1, (6, 2), 3, 2, 15, 192, 256),
    ("swiglu", "bf16", "f16", "f16", 16, (4, 4), 2, 2, 5, 256, 512),
    ("swiglu", "bf16", "f16", "int4_g32", 16, (8, 8), 1, 4, 32, 512, 384),
    ("gelu_tanh", "bf16", "f16", "none", 0, (3, 4), 1, 2, 18, 128, 192),
    ("gelu_tanh", "f32", "f32", "f32", 4, (2, 4), 1, 2, 1, 64, 128),
    ("swiglu", "f32", "f32", "f32", 12, (2, 4), 2, 4, 16, 320, 256),
    ("swiglu", "f32", "f32", "none", 0, (6, 1), 3, 1, 23, 192, 192),
    ("gelu_tanh", "f32", "f32", "f32", 16, (3, 3), 1, 1, 32, 128, 64),
    ("swiglu", "f16", "int4_g32", "int4_g32", 16, (16, 16), 2, 4, 1, 320, 192),
    ("swiglu", "f16", "int4_g32", "none", 0, (4, 4), 2, 2, 9, 256, 448),
    ("gelu_tanh", "f16", "int4_g32", "int4_g32", 9, (3, 4), 1, 3, 20, 192, 320),
    ("swiglu", "bf16", "int4_g32", "int4_g32", 16, (8, 8), 1, 4, 32, 512, 384),
    ("gelu_tanh", "bf16", "int4_g32", "none", 0, (5, 1), 2, 1, 6, 64, 64),
    ("swiglu", "bf16", "int4_g32", "int4_g32", 3, (2, 2), 2, 1, 13, 128, 192),
    # the most groups, experts and choices a layer may have
    ("swiglu", "f16", "f16", "int4_g32", 2, (16, 64), 2, 8, 32, 64, 64),
    ("swiglu", "bf16", "bf16", "none", 0, (256, 4), 8, 2, 32, 64, 64),
    ("gelu_tanh", "f32", "f32", "none", 0, (4, 256), 1, 16, 11, 64, 64),
    # input factors past 40 MB: only the chosen experts' are read, by a launch of their own
    ("swiglu", "f16", "f16", "f16", 16, (16, 64), 2, 8, 5, 704, 64),
    ("gelu_tanh", "f32", "f32", "f32", 16, (16, 64), 2, 4, 20, 704, 64),
    ("swiglu", "bf16", "bf16", "int4_g32", 16, (16, 64), 1, 8, 17, 2560, 64),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)).replace(" ", "") for c in CASES])
def test_matches_oracle(case):
    import torch
    say("[few]", case)
    w, layer, lay, X = make(*case, bias=0.0 if case[5][0] * case[5][1] >= 1024 else 0.5)
    try:
        rt = O.route(layer)
        ref = O.forward(layer, routing=rt)
        bufs = lay.route_buffers(w.T)
        for v in bufs.values():
            v.fill_(-7)
        Y = torch.full_like(X, float("nan"))
        lay.forward_few(X, Y, route_bufs=bufs)
        torch.cuda.synchronize()
        check_routing(route_to_host(bufs), rt, w, w.T)
        one = case[1] == "bf16" and case[2] != "bf16"
        e = check_y(Y, ref, w.x_dtype, one)
        say(f"[few] err {e:.2e}")
        # without routing outputs, and again: the same bits
        raw = torch.int32 if w.x_dtype == "f32" else torch.int16
        assert torch.equal(lay.forward_few(X).view(raw), Y.view(raw))
        # fewer tokens after more: nothing of the earlier pass is read
        for T in {1, w.T // 2} - {0, w.T}:
            check_y(lay.forward_few(X[:T].contiguous()), ref[:T], w.x_dtype, one)
        assert torch.equal(lay.forward_few(X).view(raw), Y.view(raw))
    finally:
        lay.close()


@pytest.mark.parametrize("wi,T", [(0, 1), (0, 32), (1, 3), (3, 9), (4, 1), (4, 32)])
def test_workload_layers(wi, T):
    """The library's own layer shapes, against the oracle and moe_forward."""
    import torch
    L = _lib()
    w, inputs, layer = make_parity_layer(WORKLOADS[wi].with_T(T))
    lay = L.Layer(L.config_from_workload(w), inputs)
    try:
        X = x_to_device(inputs["X"], w.x_dtype)
        rt = O.route(layer)
        bufs = lay.route_buffers(T)
        Y = lay.forward_few(X, route_bufs=bufs)
        torch.cuda.synchronize()
        check_routing(route_to_host(bufs), rt, w, T)
        e = check_y(Y, O.forward(layer, routing=rt), w.x_dtype, w.x_dtype == "bf16" and w.base_dtype != "bf16")
        say(f"[few] {w.name} T={T}: err {e:.2e}")
        # passes of both kinds on one handle do not disturb each other
        Yf = lay.forward(X)
        assert rel_err(y_to_host(Yf), y_to_host(Y)) <= (1e-5 if w.x_dtype == "f32" else 1e-2)
        assert torch.equal(lay.forward_few(X), Y) and torch.equal(lay.forward(X), Yf)
    finally:
        lay.close()


@pytest.mark.parametrize("bd,resid", [("f16", "f16"), ("f32", "f32"), ("int4_g32", "int4_g32"), ("f16", "none")])
@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
def test_device_weights_give_the_same_layer(bd, resid, act):
    """Weights given in device memory are packed there: the same bits as the
    host's packing, by both forward passes."""
    import torch
    xd = "f32" if bd == "f32" else "f16"
    case = (act, xd, bd, resid, 0 if resid == "none" else 16, (3, 2), 2, 1, 12, 192, 320)
    _, _, a, X = make(*case)
    _, _, b, _ = make(*case, device=True)
    try:
        assert torch.equal(a.forward_few(X), b.forward_few(X))
        if bd != "int4_g32":
            assert torch.equal(a.forward(X), b.forward(X))
    finally:
        a.close()
        b.close()


def test_weights_from_device_tensors():
    """Layer takes torch tensors as they are, bf16 among them."""
    import torch
    L = _lib()
    from compressed_expert_ffn_amd import synth
    w = workload("swiglu", "bf16", "bf16", "int4_g32", 16, (4, 4), 1, 2, 6, 256, 192)
    w, inputs, layer = make_parity_layer(w)
    dev = {}
    for key, v in inputs.items():
        if key in ("W_grp", "W_exp", "group_bias", "expert_bias"):
            dev[key] = None if v is None else torch.from_numpy(v).cuda()
        elif key in ("A", "B"):
            dev[key] = [torch.from_numpy(m).cuda() for m in v]
    dev["base"] = [torch.from_numpy(synth.bf16_bits_to_f32(b)).cuda().bfloat16() for b in inputs["base"]]
    lay = L.Layer(L.config_from_workload(w), dev, on_device=True)
    try:
        check_y(lay.forward_few(x_to_device(inputs["X"], "bf16")), O.forward(layer), "bf16")
    finally:
        lay.close()


def test_ties_and_masked_groups():
    """Equal scores go to the lower index; groups with a bias of -inf or the
    type's lowest value are left alone while others remain."""
    import torch
    L = _lib()
    from compressed_expert_ffn_amd import synth
    w = workload("swiglu", "f16", "f16", "none", 0, (6, 5), 2, 3, 4, 128, 64)
    inputs = synth.make_layer(w)
    inputs["W_grp"] = np.zeros_like(inputs["W_grp"])
    inputs["W_exp"] = np.zeros_like(inputs["W_exp"])
    for bias, want in ((None, [0, 1]), ([-np.inf, 0, -np.inf, -3.4e38, 0, -np.inf], [1, 4])):
        inputs["group_bias"] = None if bias is None else np.array(bias, dtype=np.float32)
        inputs["expert_bias"] = None
        lay = L.Layer(L.config_from_workload(w), inputs)
        bufs = lay.route_buffers(4)
        Y = lay.forward_few(x_to_device(inputs["X"], "f16"), route_bufs=bufs)
        r = route_to_host(bufs)
        assert (r["gidx"] == want).all()
        assert (r["idx"] == [g * 5 + j for g in want for j in range(3)]).all()
        assert np.abs(r["w"] - 1 / 6).max() <= 1e-6 and torch.isfinite(Y).all()
        assert (r["gcounts"] == [4 if g in want else 0 for g in range(6)]).all()
        lay.close()


@pytest.mark.parametrize("bd", ["f16", "int4_g32"])
def test_a_bad_token_spoils_only_itself(bd):
    import torch
    case = ("swiglu", "f16", bd, "int4_g32", 16, (4, 4), 2, 2, 20, 256, 192)
    w, layer, lay, X = make(*case)
    try:
        Y = lay.forward_few(X)
        bad = X.clone()
        bad[3] = float("nan")
        bad[18, 7] = float("inf")
        Yb = lay.forward_few(bad)
        keep = [t for t in range(20) if t not in (3, 18)]
        # their sums run over other groups beside theirs, so equal to rounding
        a, b = Yb[keep].double().cpu().numpy(), Y[keep].double().cpu().numpy()
        assert np.linalg.norm(a - b) <= 0.2 * STEP["f16"] * np.linalg.norm(b)
        assert not torch.isfinite(Yb[3]).any()
        bufs = lay.route_buffers(20)
        lay.forward_few(bad, route_bufs=bufs)
        r = route_to_host(bufs)
        assert (r["idx"] >= 0).all() and (r["idx"] < 16).all()
    finally:
        lay.close()


def test_no_tokens_and_refusals():
    import torch
    L = _lib()
    w, layer, lay, X = make("swiglu", "f16", "f16", "f16", 16, (4, 4), 2, 2, 8, 128, 64, T_max=40)
    try:
        bufs = lay.route_buffers(0)
        for key in ("counts", "offsets", "gcounts", "goffsets"):
            bufs[key].fill_(-7)
        assert lay.forward_few(X[:0], route_bufs=bufs).shape == (0, 128)
        torch.cuda.synchronize()
        for key in ("counts", "offsets", "gcounts", "goffsets"):
            assert (bufs[key] == 0).all()
        many = X.repeat(5, 1)[:33].contiguous()
        with pytest.raises(L.MoEError, match="few-token pass"):
            lay.forward_few(many)
        lay.forward(many)
        with pytest.raises(L.MoEError, match="T_max"):
            lay.forward_few(X.repeat(6, 1))
        with pytest.raises(ValueError, match="contiguous"):
            lay.forward_few(X.t().contiguous().t())
        with pytest.raises(ValueError, match="contiguous"):
            lay.forward_few(X.float())
        with pytest.raises(ValueError, match="Y"):
            lay.forward_few(X, torch.empty((7, 128), dtype=X.dtype, device="cuda"))
        for args in ((X.data_ptr() + 2, 1, X.data_ptr() + 512), (X.data_ptr(), 1, X.data_ptr()), (None, 1, X.data_ptr()),
                     (X.data_ptr(), 1, None), (X.data_ptr(), -1, X.data_ptr() + 512), (X.data_ptr(), 1, X.data_ptr() + 513)):
            assert L.lib.moe_forward_few(lay.h, args[0], args[1], args[2], None, None) == L.MOE_ERR_INVALID_ARG, args
        bad = lay.route_buffers(8)
        with pytest.raises(ValueError, match="idx"):
            lay.forward_few(X, route_bufs=lay.route_buffers(X.shape[0] - 1))
        for name, t in (("w", bad["w"].int()), ("counts", bad["counts"].cpu()), ("gperm", bad["gperm"][::2]),
                        ("other", bad["idx"])):
            with pytest.raises(ValueError, match=name):
                lay.forward_few(X[:8].contiguous(), route_bufs={name: t})
        lay.offload_enable(2)
        with pytest.raises(L.MoEError, match="offloaded"):
            lay.forward_few(X)
    finally:
        lay.close()


def test_a_four_bit_base_runs_nowhere_else():
    import torch
    L = _lib()
    w, layer, lay, X = make("swiglu", "bf16", "int4_g32", "int4_g32", 16, (4, 4), 2, 2, 8, 128, 64, T_max=64)
    try:
        st = lay.stats()
        base = 4 * 3 * 128 * 64
        fac = 16 * 16 * 3 * (128 + 64)
        assert st["stored_bytes"] == (base + fac) // 2 + (base + fac) // 32 * 2
        for call in (lambda: lay.forward(X), lambda: lay.forward_noalloc(X, torch.empty_like(X)),
                     lambda: lay.backward(X, X), lambda: lay.offload_enable(2)):
            with pytest.raises(L.MoEError) as e:
                call()
            assert e.value.code == L.MOE_ERR_UNSUPPORTED
        # routing alone takes any batch
        many = X.repeat(8, 1)
        r = route_to_host(lay.route(many))
        rt = O.route(layer)
        assert np.array_equal(r["idx"], np.tile(rt["idx"], (8, 1)))
        check_y(lay.forward_few(X), O.forward(layer), "bf16", True)
    finally:
        lay.close()


@pytest.mark.parametrize("case", [
    ("swiglu", "f16", "f16", "none", 0, (250, 1), 8, 1, 32, 64, 64),
    ("swiglu", "f16", "f16", "int4_g32", 3, (100, 10), 4, 4, 32, 64, 64),
    ("gelu_tanh", "bf16", "bf16", "int4_g32", 16, (17, 17), 3, 5, 24, 128, 64),
    ("swiglu", "f16", "f16", "int4_g32", 16, (1, 16), 1, 16, 32, 128, 64),
], ids=["groups", "slots", "past16", "one_group"])
def test_most_groups_and_slots(case):
    """The largest tables, more candidates than a row of lanes, a group that every token chooses."""
    import torch
    say("[few]", case)
    w, layer, lay, X = make(*case)
    try:
        rt = O.route(layer)
        bufs = lay.route_buffers(w.T)
        Y = lay.forward_few(X, route_bufs=bufs)
        torch.cuda.synchronize()
        check_routing(route_to_host(bufs), rt, w, w.T)
        check_y(Y, O.forward(layer, routing=rt), w.x_dtype)
    finally:
        lay.close()


def test_rows_behind_the_last_token_stay():
    import torch
    w, layer, lay, X = make("swiglu", "f16", "f16", "int4_g32", 16, (4, 4), 2, 2, 11, 256, 192)
    try:
        buf = torch.full((32, 256), 42.0, dtype=X.dtype, device="cuda")
        lay.forward_few(X, buf[:11])
        assert (buf[11:] == 42.0).all()
        check_y(buf[:11], O.forward(layer), "f16")
    finally:
        lay.close()


def test_repeated_passes_on_one_handle_give_equal_bits():
    """The selection's ticket returns to zero with every pass."""
    import torch
    w, layer, lay, X = make("swiglu", "f16", "f16", "int4_g32", 16, (16, 16), 2, 4, 16, 1024, 192)
    try:
        Y = lay.forward_few(X)
        outs = [lay.forward_few(X if i % 2 == 0 else X[:1 + i].contiguous()) for i in range(15)]
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i], Y) for i in range(0, 15, 2))
        check_y(Y, O.forward(layer), "f16")
    finally:
        lay.close()


@pytest.mark.parametrize("case", [
    ("swiglu", "f16", "f16", "int4_g32", 16, (16, 64), 2, 8, 32, 64, 64),
    ("swiglu", "f16", "f16", "int4_g32", 16, (8, 4), 2, 2, 9, 256, 320),
    ("gelu_tanh", "bf16", "int4_g32", "none", 0, (4, 1), 2, 1, 32, 128, 192),
    ("swiglu", "f32", "f32", "f32", 8, (4, 4), 1, 2, 3, 128, 64),
], ids=["many", "f16", "int4", "f32"])
def test_graph_replays_follow_their_input(case):
    import torch
    w, layer, lay, X0 = make(*case, bias=0.0)
    try:
        X, Y = X0.clone(), torch.empty_like(X0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            lay.forward_few(X, Y)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lay.forward_few(X, Y)
        raw = torch.int32 if w.x_dtype == "f32" else torch.int16
        for rep in range(4):
            X.copy_(X0.roll(rep, 0))
            Y.zero_()
            eager = lay.forward_few(X)
            (X.float() * 2).sum()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y.view(raw), eager.view(raw)), rep
    finally:
        lay.close()


def test_two_handles_on_two_streams():
    import torch
    cases = [("swiglu", "f16", "f16", "int4_g32", 16, (16, 4), 2, 2, 16, 1024, 512),
             ("swiglu", "bf16", "int4_g32", "none", 0, (8, 1), 2, 1, 5, 1024, 512)]
    made = [make(*c) for c in cases]
    try:
        alone = [lay.forward_few(X) for _, _, lay, X in made]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        outs = [[], []]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(6):
            for i, (_, _, lay, X) in enumerate(made):
                with torch.cuda.stream(streams[i]):
                    outs[i].append(lay.forward_few(X))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(y.view(torch.int16), alone[i].view(torch.int16)) for y in outs[i])
    finally:
        for _, _, lay, _ in made:
            lay.close()


@pytest.mark.parametrize("xd", ["f16", "bf16"])
def test_a_decode_block_of_both_operators(xd):
    """Steps of a decode loop: a 4-bit projection, the layer with a 4-bit base
    and its sum with the projection, a 4-bit output head whose best column is
    the next token.  Eager and as a captured graph; every operator against 64
    bits on the input it was given."""
    import torch
    L = _lib()
    T, d, vocab = 3, 256, 67
    w, layer, lay, X0 = make("swiglu", xd, "int4_g32", "int4_g32", 16, (4, 4), 2, 2, T, d, 192)
    rng = np.random.default_rng(7)

    def linear(n_out):
        q = rng.integers(-8, 8, (d, n_out)).astype(np.int8)
        scale = np.full((d // 64, n_out), 1 / (4.6 * np.sqrt(d)), np.float16)
        ref = q * np.repeat(scale.astype(np.float64), 64, axis=0)
        return L.QuantLinear(d, n_out, 64, xd, q=q, scale=scale), ref

    (proj, Wp), (head, Wh) = linear(d), linear(vocab)
    try:
        emb = torch.from_numpy(rng.standard_normal((vocab, d)).astype(np.float32)).cuda().to(X0.dtype)
        X = torch.empty_like(X0)
        H, M, Z = torch.empty_like(X0), torch.empty_like(X0), torch.empty((T, vocab), dtype=X0.dtype, device="cuda")

        def step():
            proj.matvec(X, H)
            lay.forward_few(H, M)
            M.add_(H)
            head.matvec(M, Z)

        def run(call):
            tok, seen = torch.tensor([5, 40, 66], device="cuda"), []
            for _ in range(4):
                X.copy_(emb[tok])
                call()
                tok = Z.argmax(1)
                seen.append([t.clone() for t in (X, H, M, Z, tok)])
            torch.cuda.synchronize()
            return seen

        eager = run(step)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for a, b in zip(eager, run(g.replay)):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        for x, h, m, z, _ in eager:
            x, m = y_to_host(x), y_to_host(m)
            hd = y_to_host(h)
            check_y(h, x @ Wp, xd)
            host = h.cpu().view(torch.int16).numpy()
            moe = O.forward(dict(layer, X=host.view(np.float16) if xd == "f16" else host.view(np.uint16)))
            # the layer's result and the sum are each rounded once
            ref = moe + hd
            assert (np.abs(m - ref) <= STEP[xd] * (np.abs(moe) * 1.05 + np.abs(ref) * 1.05 + 0.05 *
                                                   np.abs(moe).max())).all()
            check_y(z, m @ Wh, xd)
    finally:
        proj.close()
        head.close()
        lay.close()
