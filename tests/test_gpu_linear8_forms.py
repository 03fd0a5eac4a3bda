"""Every form of the 8-bit products' kernels by its plan: stream-K, panels cut along N,
wide streaming blocks and the two products of a binary32 gradient; and the calls from
threads, under another current stream and without the C extension."""
import threading

import pytest
import torch

import linear8_cases as cases
import linear8_ref as ref
import test_gpu_linear8 as layer
from gpu_util import need_gpu
from linear8_ref import DT, SUB, U, U32

pytestmark = pytest.mark.gpu


def put(t, stride, offset=0):
    """A device copy of t whose rows lie `stride` elements apart, with NaN patterns between."""
    v = ref.strided(t.shape[0], t.shape[1], stride - t.shape[1], t.dtype, "cuda", offset)
    v.copy_(t)
    return v


def workspace(nbytes):
    """nbytes of workspace (NaN patterns) and a guard behind it, or none."""
    return torch.full((nbytes + 4096,), 0x7F, dtype=torch.uint8, device="cuda") if nbytes else None


def untouched(ws, nbytes):
    return ws is None or bool((ws[nbytes:] == 0x7F).all())


def rows_to_check(M):
    return sorted({0, min(1, M - 1), M - 1, max(M - 2, 0), *range(5, M, max(1, M // 40))})


@pytest.mark.parametrize("case", cases.SCALED, ids=str)
def test_scaled_forms(case):
    mcg = need_gpu()
    layout, M, N, K, aligned, nb, kernel, panels, streamk, ranges = case
    lda, ldb = cases.scaled_lds(layout, M, N, K, aligned)
    a, b = ref.codes(K, M, K), ref.codes(K + 1, K, N)
    sa, sb, bias = ref.rand(1, M).abs().float() + 0.1, ref.rand(2, N).abs().float() + 0.1, 1e4 * ref.rand(3, N).float()
    A, B = put(a, lda), put(b.T.contiguous() if layout == "k_contig" else b, ldb)
    ws = workspace(nb)
    got, p = mcg.i8_scaled_path(layout, M, N, K, A, lda, B, ldb, nb)
    assert (got, p["streamk_tiles"], p["ranges"]) == (kernel, streamk, ranges) and p["workspace"] <= nb
    rows = rows_to_check(M)
    core = ref.i8_scaled(a[rows], sa[rows], b, sb, None)
    for dt, use_bias, pad in (("f32", True, 0), ("bf16", False, 3), ("f16", True, 4)):
        scale = 1e-6 if dt == "f16" else 1.0  # (within f16's range)
        ga, gb, gc = sa.cuda(), (sb * scale).cuda(), (bias * scale).cuda() if use_bias else None
        D = layer.empty(M, N, DT[dt], pad)
        mcg.gemm_i8_scaled(layout, M, N, K, A, lda, ga, B, ldb, gb, gc, D, N + pad, dt, ws, nb)
        layer.guards_hold(D)
        assert untouched(ws, nb)
        exact = ref.i8_scaled(a[rows], sa[rows], b, gb.cpu(), None)
        d = exact + gc.cpu().double() if use_bias else exact
        layer.within(D[rows], d, layer.scaled_tol(d, exact, gc, dt), f"{dt} {case}")
        # the sums are exact: every form gives the bits of the one without a workspace
        base = layer.empty(M, N, DT[dt], pad)
        mcg.gemm_i8_scaled(layout, M, N, K, A, lda, ga, B, ldb, gb, gc, base, N + pad, dt)
        assert torch.equal(D, base)
    assert core.abs().max() > 0


def grad_call(mcg, dt, case, A, lda, Q, s, C, D, beta, ws):
    dtD, layout, M, N, K, aligned, nb, *_ = case
    mcg.gemm_grad_i8(dt, layout, M, N, K, A, lda, Q, N, s, C, D, D.stride(0), "f32" if dtD == "f32" else dt, beta, ws, nb)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("case", cases.GRAD, ids=str)
def test_gradient_forms(case, dt):
    mcg = need_gpu()
    dtD, layout, M, N, K, aligned, nb, kernel, panels, streamk = case
    out = "f32" if dtD == "f32" else dt
    lda = cases.grad_lda(layout, M, K, aligned)
    a = ref.rand(K, M, K).to(DT[dt])
    q, s = cases.grad_inputs(K + 1, K, N)
    A, Q, S = put(a if layout == "k_contig" else a.T.contiguous(), lda), put(q, N), s.cuda()
    ws = workspace(nb)
    got, p = mcg.grad_i8_path(dt, layout, M, N, K, A, lda, Q, N, out, nb)
    assert (got, p["streamk_tiles"]) == (kernel, streamk) and p["workspace"] <= nb
    rows = rows_to_check(M)
    core, mag = ref.grad_i8(a[rows], q, s, None, 0.0)
    c = ref.rand(K + 3, M, N).to(DT[out])
    for beta, pad in ((0.0, 0), (-0.5, 4), (1.0, 3)):
        C, D = put(c, N + pad), layer.empty(M, N, DT[out], pad)
        grad_call(mcg, dt, case, A, lda, Q, S, C if beta else None, D, beta, ws)
        layer.guards_hold(D)
        assert untouched(ws, nb) and torch.equal(C.cpu(), c)
        d = core + beta * c[rows].double()
        full = mag + abs(beta) * c[rows].double().abs()
        layer.within(D[rows], d, layer.grad_tol(dt, out, a[rows], s, d, full, K), f"{dt} -> {out} {case} beta {beta}")
        assert bool(torch.isfinite(D).all())
        if beta:  # D may be C
            grad_call(mcg, dt, case, A, lda, Q, S, C, C, beta, ws)
            torch.cuda.synchronize()
            assert torch.equal(C, D)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("case", [c for c in cases.GRAD if c[0] == "f32"], ids=str)
def test_binary32_gradients_hold_the_rest_of_the_rounding(case, dt):
    # few nonzeros a row, so that the sum's own bound does not hide the second value of s q
    mcg = need_gpu()
    dtD, layout, M, N, K, aligned, nb, kernel, panels, streamk = case
    n = 4
    lda = cases.grad_lda(layout, M, K, aligned)
    a = cases.few_nonzeros(K, M, K, n, dt)
    q, s = cases.grad_inputs(K + 1, K, N)
    A, Q = put(a if layout == "k_contig" else a.T.contiguous(), lda), put(q, N)
    ws = workspace(nb)
    D = layer.empty(M, N, torch.float32)
    grad_call(mcg, dt, case, A, lda, Q, s.cuda(), None, D, 0.0, ws)
    torch.cuda.synchronize()
    rows = rows_to_check(M)
    d, mag = ref.grad_i8(a[rows], q, s, None, 0.0)
    layer.within(D[rows], d, cases.sparse_grad_tol(dt, a[rows], d, mag, n), f"{dt} {case}")


# ------------------------------------------- streams, threads and the binding
def snapshot(s):
    torch.cuda.synchronize()
    return {k: s[k].clone() for k in layer.OUTS}


def reset(s):
    for k in layer.OUTS:
        s[k].fill_(-77 if s[k].dtype == torch.int8 else float("nan"))
    torch.cuda.synchronize()


def same(s, want, what):
    torch.cuda.synchronize()
    for k in layer.OUTS:
        assert torch.equal(s[k].contiguous().view(torch.uint8), want[k].contiguous().view(torch.uint8)), f"{what}: {k}"


def test_the_current_stream_is_the_one_of_the_context():
    # stream=None under torch.cuda.stream(...): the calls are captured from that stream
    mcg = need_gpu()
    T, K, N = 37, 512, 336
    s = layer.layer_state(T, K, N)
    layer.layer_step(mcg, s, T, K, N)
    eager = snapshot(s)
    st = torch.cuda.Stream()
    reset(s)
    with torch.cuda.stream(st):
        layer.layer_step(mcg, s, T, K, N)
    st.synchronize()
    same(s, eager, "under another current stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        layer.layer_step(mcg, s, T, K, N)
    for rep in range(3):
        reset(s)
        g.replay()
        same(s, eager, f"replay {rep}")
    reset(s)
    layer.layer_step(mcg, s, T, K, N)
    same(s, eager, "on the default stream again")


def test_threads_with_a_stream_each():
    mcg = need_gpu()
    shapes = [(37, 512, 336), (130, 768, 256), (1, 1024, 512)]
    states = [layer.layer_state(*sh) for sh in shapes]
    want = []
    for s, sh in zip(states, shapes):
        layer.layer_step(mcg, s, *sh)
        want.append(snapshot(s))
        reset(s)
    errors = []
    start = threading.Barrier(len(shapes))

    def work(i):
        try:
            st = torch.cuda.Stream()
            start.wait(30)
            with torch.cuda.stream(st):  # (a thread's current stream is its own)
                for _ in range(20):
                    layer.layer_step(mcg, states[i], *shapes[i])
            st.synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and not any(t.is_alive() for t in threads), errors
    for s, w, sh in zip(states, want, shapes):
        same(s, w, str(sh))


def test_the_calls_through_ctypes_are_the_same(monkeypatch):
    mcg = need_gpu()
    T, K, N = 37, 500, 333
    s = layer.layer_state(T, K, N)
    layer.layer_step(mcg, s, T, K, N)
    want = snapshot(s)
    q = ref.rand(1, T, K).to(torch.bfloat16).cuda()
    Q, sc, D = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, K, device="cuda")
    mcg.quantize_rows("bf16", T, K, q, K, Q, K, sc)
    mcg.dequantize_rows("f32", T, K, Q, K, sc, D, K)
    torch.cuda.synchronize()
    base = Q.clone(), sc.clone(), D.clone()
    monkeypatch.setattr(mcg, "_mcgcall", mcg._CtypesCalls())
    for st in (None, torch.cuda.Stream()):
        reset(s)
        layer.layer_step(mcg, s, T, K, N, stream=st)
        same(s, want, f"through ctypes on {st}")
    for t in (Q, sc, D):
        t.zero_()
    mcg.quantize_rows("bf16", T, K, q, K, Q, K, sc)
    mcg.dequantize_rows("f32", T, K, Q, K, sc, D, K)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((Q, sc, D), base))
