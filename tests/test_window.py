"""Sliding-window attention with sink tokens (attn_fwd_window, attn_bwd_window) against the definition in 64 bits:
windows of one key up to the whole sequence, windows and sinks that end inside, at and past a 128-key tile, both
alignments, ragged lengths, grouped heads, rows without keys, and key tiles with sinks whose backward work is cut
into chunks, by heads too where there are few.

Tolerances are those of the dense entry points: |dO| <= 1e-2 and |dLSE| <= 1e-3 (parity_util: an output of
magnitude below 4 is rounded to bf16 by at most 2^-7, P by 2^-12 of itself), and for a gradient the rounding of its
exact value plus 1e-2 of its tensor's largest one (test_backward: P and dS are rounded to bf16, 2^-9 of each term).
"""
import numpy as np
import pytest
import torch

from attention_forward_06_gb300 import _lib, ops
from attention_forward_06_gb300.inputs import draw
from parity_util import compare
from plain_attention import backward, forward, window_mask
from test_backward import check

CASES = [
    # B, Hq, Hkv, Sq, Sk, D, causal, window, sinks
    (1, 2, 1, 300, 300, 128, 1, 1, 0),         # each row sees itself alone
    (1, 2, 2, 300, 300, 64, 1, 1, 1),
    (1, 4, 2, 513, 513, 128, 1, 127, 0),
    (2, 4, 1, 513, 513, 64, 1, 128, 4),
    (1, 2, 1, 700, 700, 128, 1, 129, 128),     # sinks end at a tile's edge
    (1, 3, 3, 700, 700, 64, 1, 130, 130),      # sinks reach into a second tile
    (1, 8, 2, 257, 1500, 128, 1, 300, 4),      # a chunk against its context
    (1, 8, 2, 1, 1000, 128, 1, 100, 2),        # one row
    (1, 2, 1, 600, 200, 128, 1, 50, 3),        # Sq > Sk bottom-right: rows without keys
    (1, 2, 1, 900, 200, 64, 2, 60, 0),         # top-left, rows past every window: no keys
    (1, 2, 1, 900, 200, 128, 2, 60, 7),        # the same rows see the sinks alone
    (1, 2, 2, 200, 900, 64, 2, 33, 1),         # keys no row sees
    (1, 2, 1, 2500, 2500, 128, 1, 5, 3),       # the sinks' tile in chunks
    (1, 4, 1, 2500, 2600, 64, 1, 200, 260),    # three tiles with sinks, each in chunks, cut by heads too
    (1, 3, 3, 2500, 2500, 128, 1, 5, 3),       # chunks alone: one head per kv head
    (1, 6, 1, 800, 800, 128, 1, 150, 0),       # cut by heads alone
    (1, 9, 1, 4500, 4500, 64, 1, 700, 0),      # ... into groups of which the last is shorter
    (1, 4, 2, 900, 900, 128, 1, 100, 16),      # as many sinks as a step of few keys holds, and one more
    (1, 4, 2, 900, 900, 64, 1, 100, 17),
    (1, 3, 1, 900, 900, 64, 1, 300, 16),       # three heads of a group: 256 rows of each
    (1, 2, 1, 300, 300, 128, 1, 10 ** 9, 0),   # the window holds everything
    (1, 2, 1, 300, 300, 64, 1, 20, 10 ** 9),   # every key is a sink
    (1, 1, 1, 1, 1, 64, 2, 1, 0),
]
IDS = lambda c: "x".join(map(str, c))  # noqa: E731


def scale_of(D):
    return float(np.float32(D ** -0.5))


def run_forward(q, k, v, causal, window, sinks, scale):
    o, lse = ops.attn_fwd_window(q.cuda(), k.cuda(), v.cuda(), window, sinks=sinks, causal=causal, scale=scale)
    st, site = ops.debug_status()
    assert st == ops.ATTN_OK, f"kernel wait ran out at site {site}"
    return o, lse


def run_backward(q, k, v, o, lse, do, causal, window, sinks, scale):
    g = ops.attn_bwd_window(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), window, sinks=sinks, causal=causal,
                            scale=scale)
    st, site = ops.bwd_debug_status()
    assert st == ops.ATTN_OK, f"backward wait ran out at site {site}"
    return g


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_and_backward_match_the_definition(case):
    B, Hq, Hkv, Sq, Sk, D, causal, window, sinks = case
    q, k, v = draw(B, Hq, Hkv, Sq, Sk, D, seed=Sq + Sk + sinks)
    do = draw(B, Hq, Hkv, Sq, Sk, D, seed=Sq + Sk + sinks + 1)[0]
    scale, vis = scale_of(D), window_mask(Sq, Sk, causal, window, sinks)
    o, lse = run_forward(q, k, v, causal, window, sinks, scale)
    compare(o, lse, *forward(q, k, v, vis, scale))
    grads = run_backward(q, k, v, o, lse, do, causal, window, sinks, scale)
    one_key = vis.sum(1).max() == 1
    for name, g, ref in zip(("dq", "dk", "dv"), grads, backward(q, k, v, do, vis, scale)):
        if one_key and name != "dv":
            # dS = dP - D_i vanishes: what is left is the rounding of two fp32 sums of D products, each at most
            # D 2^-24 of the sum of their magnitudes, times scale and the other factor (q sums over a group's heads)
            sums = do.double().abs().reshape(-1, D) @ v.double().abs().reshape(-1, D).T
            factor = (k if name == "dq" else q).double().abs().max() * (1 if name == "dq" else Hq // Hkv)
            assert np.abs(ref).max() < 1e-12
            assert g.double().abs().max().item() <= (2 * D * 2 ** -24 * sums.max() * factor * scale).item()
        else:
            check(name, g.cpu(), ref)


@pytest.mark.gpu
def test_sharp_logits_move_the_reference_value():
    # sinks far below and far above the window's logits: the running reference moves both ways
    for factor in (0.02, 12.0):
        q, k, v = draw(1, 2, 1, 700, 700, 128, seed=5, qk_std=2.0)
        k[:, :, :4] *= factor
        scale, vis = scale_of(128), window_mask(700, 700, 1, 200, 4)
        o, lse = run_forward(q, k, v, 1, 200, 4, scale)
        compare(o, lse, *forward(q, k, v, vis, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_a_window_over_everything_is_the_dense_call_bitwise(D):
    for Hkv, causal in ((2, 1), (2, 2), (4, 1), (4, 2)):
        q, k, v = [t.cuda() for t in draw(2, 4, Hkv, 700, 900, D, seed=23)]
        do = draw(2, 4, Hkv, 700, 900, D, seed=24)[0].cuda()
        dense = ops.attn_fwd(q, k, v, causal=causal)
        near = ops.attn_fwd_window(q, k, v, 900, causal=causal)
        assert all(torch.equal(a, b) for a, b in zip(dense, near))
        if Hkv == 2:  # so few items are cut by heads, and the heads' sums are added in another order
            continue
        a = ops.attn_bwd(q, k, v, *dense, do, causal=causal)
        b = ops.attn_bwd_window(q, k, v, *near, do, 900, causal=causal)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_so_many_sinks_that_their_tiles_are_not_cut_are_the_dense_call_bitwise():
    # 33 tiles with sinks in each of 64 kv slices: one item each, whose query tiles come in the dense call's order
    q, k, v = [t.cuda() for t in draw(32, 2, 2, 4224, 4224, 64, seed=25)]
    do = draw(32, 2, 2, 4224, 4224, 64, seed=26)[0].cuda()
    o, lse = ops.attn_fwd(q, k, v, causal=1)
    a = ops.attn_bwd(q, k, v, o, lse, do, causal=1)
    b = ops.attn_bwd_window(q, k, v, o, lse, do, 1, sinks=4224)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_keys_out_of_every_window_do_not_matter():
    # K rows that no row sees hold infinities and NaN, in tiles that are loaded for their other keys
    q, k, v = draw(1, 2, 1, 100, 1000, 128, seed=31)
    o, lse = run_forward(q, k, v, 1, 50, 2, scale_of(128))
    bad = k.clone()
    bad[:, :, 2:851] = float("nan")
    bad[:, :, 2:851:3] = float("inf")
    o2, lse2 = run_forward(q, bad, v, 1, 50, 2, scale_of(128))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_gradients_against_differences():
    """The derivative of sum(O dO) along a random direction, from the plain forward in 64 bits, against the kernel's
    gradients: the sum of n products whose factors carry a relative error of about 2^-8 each (bf16 gradients, P and
    dS), so within 2^-8 of the products' 2-norm times four."""
    B, Hq, Hkv, Sq, Sk, D, causal, window, sinks = 1, 4, 2, 260, 300, 64, 1, 70, 5
    q, k, v = draw(B, Hq, Hkv, Sq, Sk, D, seed=91)
    do = draw(B, Hq, Hkv, Sq, Sk, D, seed=92)[0]
    scale, vis = scale_of(D), window_mask(Sq, Sk, causal, window, sinks)
    o, lse = run_forward(q, k, v, causal, window, sinks, scale)
    grads = run_backward(q, k, v, o, lse, do, causal, window, sinks, scale)
    for at, g in enumerate(grads):
        g = g.cpu().double()
        step = torch.randn(g.shape, generator=torch.Generator().manual_seed(at), dtype=torch.float64)
        eps, side = 1e-4, []
        for sign in (1, -1):
            x = [t.double() for t in (q, k, v)]
            x[at] = x[at] + sign * eps * step
            side.append((forward(*x, vis, scale)[0] * do.double().numpy()).sum())
        terms = g * step
        assert abs((side[0] - side[1]) / (2 * eps) - terms.sum().item()) <= 4 * 2 ** -8 * terms.norm().item()


@pytest.mark.gpu
def test_in_a_graph_and_on_another_stream():
    shape = (1, 4, 2, 600, 2600, 128)
    first, second = [[t.cuda() for t in draw(*shape, seed=s)] for s in (41, 43)]
    do = draw(*shape, seed=45)[0].cuda()

    def calls(q, k, v):
        o, lse = ops.attn_fwd_window(q, k, v, 200, sinks=4)
        return (o, lse, *ops.attn_bwd_window(q, k, v, o, lse, do, 200, sinks=4))

    want = [[t.clone() for t in calls(*x)] for x in (first, second)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls(*first)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    static = [t.clone() for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(*static)
    for data, ref in ((second, want[1]), (first, want[0])):
        for dst, src in zip(static, data):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 8, 2, 500, 64, 100, 4), (2, 8, 8, 1000, 64, 200, 0), (1, 16, 1, 900, 128, 60, 20)],
                         ids=IDS)
def test_calls_back_to_back_are_calls_one_by_one(shape):
    # a call starts under the kernel before it, which here writes what it reads: q, k, v and dO of each step come from
    # kernels right before it, and the backward follows its forward at once
    B, Hq, Hkv, S, D, window, sinks = shape

    def run(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        base = [t.cuda() for t in draw(B, Hq, Hkv, S, S, D, seed=61)]
        do = draw(B, Hq, Hkv, S, S, D, seed=62)[0].cuda()
        outs = []
        for step in range(6):
            q, k, v, g = (t * (1.0 + 0.125 * step) for t in (*base, do))
            pause()
            o, lse = ops.attn_fwd_window(q, k, v, window, sinks=sinks)
            pause()
            outs += [o, lse, *ops.attn_bwd_window(q, k, v, o, lse, g, window, sinks=sinks)]
            pause()
        torch.cuda.synchronize()
        return outs

    slow = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(slow, run(False)))


@pytest.mark.gpu
def test_empty_sequences():
    q, k, v = [t.cuda() for t in draw(1, 2, 1, 64, 64, 128, seed=43)]
    o, lse = ops.attn_fwd_window(q, k[:, :, :0].contiguous(), v[:, :, :0].contiguous(), 4)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    none = q[:, :, :0].contiguous()
    dq, dk, dv = ops.attn_bwd_window(none, k, v, none, torch.zeros((1, 2, 0), device="cuda"), none, 4, sinks=2,
                                     dk=torch.full_like(k, 7.0), dv=torch.full_like(v, 7.0))
    assert dq.numel() == 0 and torch.all(dk == 0) and torch.all(dv == 0)


# ---------------------------------------------------------------------------- on the CPU
def test_the_plain_gradients_against_differences():
    q, k, v = [t.double() for t in draw(1, 2, 1, 9, 12, 64, seed=3)]
    do = draw(1, 2, 1, 9, 12, 64, seed=4)[0].double()
    for causal, window, sinks in ((1, 3, 2), (2, 4, 0), (1, 1, 0)):
        vis = window_mask(9, 12, causal, window, sinks)
        for at, g in enumerate(backward(q, k, v, do, vis, 0.125)):
            step = torch.randn(g.shape, generator=torch.Generator().manual_seed(at), dtype=torch.float64)
            loss = []
            for sign in (1, -1):
                x = [q, k, v]
                x[at] = x[at] + sign * 1e-5 * step
                loss.append((forward(*x, vis, 0.125)[0] * do.numpy()).sum())
            assert abs((loss[0] - loss[1]) / 2e-5 - (g * step.numpy()).sum()) < 1e-6


def test_window_mask_by_hand():
    rows = ["".join("x" if c else "." for c in r) for r in window_mask(4, 6, 1, 2, 1)]
    assert rows == ["xxx...", "x.xx..", "x..xx.", "x...xx"]
    rows = ["".join("x" if c else "." for c in r) for r in window_mask(5, 2, 2, 2, 0)]
    assert rows == ["x.", "xx", ".x", "..", ".."]


Q, K, V, O, L = 0x100000, 0x200000, 0x300000, 0x400000, 0x500000  # never read: the checks come first


@pytest.mark.parametrize("kw", [dict(causal=0), dict(causal=3), dict(window=0), dict(window=-1), dict(sinks=-1),
                                dict(D=96), dict(Hq=3), dict(scale=0.0), dict(scale=float("nan")), dict(Sq=-1)])
def test_invalid_arguments(kw):
    a = dict(dict(B=1, Hq=4, Hkv=2, Sq=64, Sk=64, D=128, causal=1, window=8, sinks=2, scale=0.1), **kw)
    tail = (a["B"], a["Hq"], a["Hkv"], a["Sq"], a["Sk"], a["D"], a["causal"], a["window"], a["sinks"], a["scale"])
    assert _lib.load().attn_fwd_window(Q, K, V, O, L, *tail, None) == ops.ATTN_ERR_INVALID_ARG
    assert _lib.load("attn_bwd").attn_bwd_window(Q, K, V, O, L, 0x600000, 0x700000, 0x800000, 0x880000, *tail,
                                                 0x900000, 1 << 30, None) == ops.ATTN_ERR_INVALID_ARG


def test_pointers_and_workspace():
    fwd = lambda q=Q, o=O: _lib.load().attn_fwd_window(q, K, V, o, L, 1, 4, 2, 64, 64, 128, 1, 8, 2, 0.1,  # noqa: E731
                                                       None)
    assert fwd(q=0) == ops.ATTN_ERR_NULL_PTR
    assert fwd(o=O + 4) == ops.ATTN_ERR_MISALIGNED
    assert fwd(o=K) == ops.ATTN_ERR_INVALID_ARG
    lib = _lib.load("attn_bwd")
    need = ops.bwd_window_workspace_size(1, 4, 4, 2500, 2500, 128, 5, 3)
    # -LSE and -D of 2560 rows of four heads, then dV and dK of the one tile with sinks: 5 chunks of 4 query tiles
    assert need == 2 * 4 * 2560 * 4 + 5 * 4 * 2 * 128 * 128 * 4
    # two heads per kv head: each of the 24 items of a kv head is cut in two
    need = ops.bwd_window_workspace_size(1, 4, 2, 2500, 2500, 128, 5, 3)
    assert need == 2 * 4 * 2560 * 4 + 2 * 24 * 2 * 2 * 128 * 128 * 4
    bwd = lambda ws=0x9000000, n=need: lib.attn_bwd_window(  # noqa: E731
        0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x5000000, 0x6000000, 0x7000000, 0x8000000, 0x8800000, 1, 4, 2,
        2500, 2500, 128, 1, 5, 3, 0.1, ws, n, None)
    assert bwd(n=need - 1) == ops.ATTN_ERR_INVALID_ARG
    assert bwd(ws=0) == ops.ATTN_ERR_NULL_PTR
    assert bwd(ws=0x7000000) == ops.ATTN_ERR_INVALID_ARG  # over dq
    # many sinks: at most 1024 partials of dV and dK
    for sinks in (1024, 4096, 32768, 2 ** 31 - 1):
        size = ops.bwd_window_workspace_size(1, 32, 8, 32768, 32768, 128, 1024, sinks)
        assert 0 <= size - 2 * 32 * 32768 * 4 <= 1024 * 2 * 128 * 128 * 4
    for bad in (dict(window=0), dict(sinks=-1), dict(D=96), dict(Hkv=0), dict(Hkv=3)):
        a = dict(dict(B=1, Hq=4, Hkv=2, Sq=64, Sk=64, D=128, window=8, sinks=2), **bad)
        assert lib.attn_bwd_window_workspace_size(*a.values()) == 0


def test_the_binding_refuses_what_is_not_a_cuda_tensor():
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.attn_fwd_window(q, q, q, 4)
