"""GPU parity of the whole-layer call (up to 32 tokens, one launch) against the layer's definition in 64 bits.

Tolerance of fp32 outputs, per token in the 2-norm.  A projection's result is a sum over G groups of s (sum q u) +
b (sum u).  Its fp32 roundings: four MMA blocks per group (each truncating against its largest addend: charged 34
units of 2^-24, see parity.tc_chain_rounds), two multiply-adds per group, up to 16 partial sums: about n = 220 in a
chain.  They fall on partial sums whose size is that of the unsigned code sums, at most 4 times (codes 0..15 about their
middle 7.5 with deviation 4.6, bias of the same size) that of the result for inputs of random sign, and add up like
sqrt(n): sqrt(220) * 2^-24 * 4 = 3.5e-6.  Two projections and SwiGLU (which passes at most 1.1 of its input's relative
error on each factor, and rounds h to 22 bits) follow one another: 3 * 3.5e-6 = 1.1e-5.
"""
import numpy as np
import pytest
import torch

import int4_expert_ffn_top_b200 as M
from int4_expert_ffn_top_b200 import _lib
from parity import EPS32, check_topk, tc_chain_rounds

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPSBF = torch.finfo(torch.bfloat16).eps / 2
OUT_TOL = 1.1e-5
EPS = 1e-6


# ----------------------------------------------------------------------------- layers and their definition
def records(g, rows, n_in, bits, scale=1.0):
    cb, G = n_in * bits // 8, n_in // 64
    rec = torch.randint(0, 256, (*rows, M.qrow_bytes(n_in, bits)), dtype=torch.uint8, device=DEV, generator=g)
    s = (torch.rand((*rows, G), device=DEV, generator=g) * 0.015 + 0.005) * scale / (1 if bits == 4 else 16)
    s = s.half()
    b = (-(2.0 ** (bits - 1) + torch.randn((*rows, G), device=DEV, generator=g) * 2.0 ** (bits - 6)) * s.float()).half()
    rec[..., cb:cb + 2 * G] = s.view(torch.uint8)
    rec[..., cb + 2 * G:cb + 4 * G] = b.view(torch.uint8)
    return rec


def blocks(g, n, H, I, scale=1.0):
    gu, dn = records(g, (n, 2 * I), H, 4, scale).view(n, -1), records(g, (n, H), I, 4, scale).view(n, -1)
    out = torch.randint(0, 256, (n, M.block_stride(H, I)), dtype=torch.uint8, device=DEV, generator=g)
    out[:, :gu.shape[1]] = gu
    out[:, gu.shape[1]:gu.shape[1] + dn.shape[1]] = dn
    return out


class Layer:
    """Random layer in the storage formats; sh: which of the shared expert's adapters exist."""

    def __init__(self, H, E, I, r=0, sh=(True, True, True), down=False, gate_up=False, bias=0.5, seed=0, scale=1.0,
                 lora_scale=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed * 7919 + H + E + I + r)
        self.H, self.E, self.I, self.r, self.ls = H, E, I, r, lora_scale

        def ad(n, n_in, n_out):
            return ((torch.randn((*n, r, n_in), device=DEV, generator=g) * 0.05).half(),
                    (torch.randn((*n, n_out, r), device=DEV, generator=g) * 0.05).half())

        self.router, self.gate = records(g, (E,), H, 8), records(g, (1,), H, 8)
        self.bias = torch.randn(E, device=DEV, generator=g) * bias
        self.pool, self.shared = blocks(g, E, H, I, scale), blocks(g, 1, H, I, scale)[0]
        self.sh = [ad((), *d) if r and on else None for on, d in zip(sh, ((H, I), (H, I), (I, H)))]
        self.down = ad((E,), I, H) if r and down else None
        self.gu = None
        if r and gate_up:
            self.gu = ((torch.randn((E, 2, r, H), device=DEV, generator=g) * 0.05).half(),
                       (torch.randn((E, 2 * I, r), device=DEV, generator=g) * 0.05).half())
        self.dev = M.DeviceLayer.from_tensors(
            H=H, E=E, I=I, r=r, router=self.router, router_bias=self.bias, shared_gate=self.gate,
            shared_block=self.shared, pool=self.pool, shared_lora=self.sh if r else None, routed_down_lora=self.down,
            routed_gate_up_lora=self.gu, lora_scale=lora_scale)


def matrix(rec, n_in, bits):
    at = torch.arange(n_in, device=rec.device)
    if bits == 4:
        q = (rec[:, at // 2].long() >> (4 * (at % 2))) & 15
    else:
        q = rec[:, at].long()
    tail = rec[:, n_in * bits // 8:].contiguous().view(torch.float16).double()
    return q * tail[:, at // 64] + tail[:, n_in // 64 + at // 64]


def ffn(L, block, u, gate=None, up=None, down=None):
    cut = 2 * L.I * M.qrow_bytes(L.H, 4)
    W = matrix(block[:cut].view(2 * L.I, -1), L.H, 4)
    Dn = matrix(block[cut:cut + L.H * M.qrow_bytes(L.I, 4)].view(L.H, -1), L.I, 4)

    def delta(p, v):
        return 0.0 if p is None else L.ls * ((v @ p[0].double().T) @ p[1].double().T)

    a, b = u @ W[0::2].T + delta(gate, u), u @ W[1::2].T + delta(up, u)
    h = a * torch.sigmoid(a) * b
    return h @ Dn.T + delta(down, h)


def normed(x):
    x = x.double()
    return (x / (x.square().mean(1, keepdim=True) + EPS).sqrt()).float().bfloat16()


def definition(L, u, K, executed=None):
    """(logits, idx, w, out) in 64 bits for bf16 u."""
    u = u.double()
    logits = u @ matrix(L.router, L.H, 8).T + L.bias.double()
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :K]
    ex = idx if executed is None else executed.long().clamp(0, L.E - 1)
    w = torch.softmax(torch.gather(logits, 1, ex), 1)
    out = torch.sigmoid(u @ matrix(L.gate, L.H, 8).T) * ffn(L, L.shared, u, *L.sh)
    for e in torch.unique(ex).tolist():
        t, k = torch.nonzero(ex == e, as_tuple=True)
        dn = None if L.down is None else (L.down[0][e], L.down[1][e])
        g = up = None
        if L.gu is not None:
            g, up = (L.gu[0][e, 0], L.gu[1][e, 0::2]), (L.gu[0][e, 1], L.gu[1][e, 1::2])
        out.index_put_((t,), w[t, k][:, None] * ffn(L, L.pool[e], u[t], g, up, dn), accumulate=True)
    return logits, idx, w, out


class Call:
    def __init__(self, L, T, K, mode=M.OUT_F32, offset=0):
        self.L, self.T, self.K, self.mode = L, T, K, mode
        self.idx = torch.full((T, K), -1, dtype=torch.int32, device=DEV)
        self.w = torch.full((T, K), float("nan"), device=DEV)
        self.logits = torch.full((T, L.E), float("nan"), device=DEV)
        self.buf = torch.full((T * L.H + 64 + offset,), 7.0, device=DEV,
                              dtype=torch.bfloat16 if mode == M.OUT_BF16 else torch.float32)
        self.out = self.buf[offset:offset + T * L.H].view(T, L.H)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = M.workspace(M.moe_layer_decode_workspace_size(L.dev, T, K))
        self.ws.fill_(0xA5)  # contents on entry must not matter

    def __call__(self, u=None, x=None, executed=None, out=None, logits=True):
        M.moe_layer_decode(self.L.dev, u, self.K, self.idx, self.w, self.out if out is None else out, self.mode, self.ws,
                           x=x, eps=EPS, exec_idx=executed, logits=self.logits if logits else None, err_word=self.err)
        return self


def rel(a, b):
    return ((a.double() - b).norm(dim=1) / b.norm(dim=1)).max().item()


def logit_tau(L, u):
    """Bound on the fp32 logits: per group four MMA blocks on each of the even and odd inputs, two multiply-adds and
    the odd half's join, 16 partial sums, the bias."""
    G = L.H // 64
    at = torch.arange(L.H, device=DEV)
    tail = L.router[:, L.H:].contiguous().view(torch.float16).double().abs()
    mag = L.router[:, :L.H].double() * tail[:, at // 64] + tail[:, G + at // 64]
    n = tc_chain_rounds(4) + 3 * G + 16 + 8
    return (n * EPS32 * (u.double().abs() @ mag.T) + 4 * EPS32 * L.bias.abs().double()).cpu().numpy()


def check(c, u, executed=None, base=None):
    torch.cuda.synchronize()
    assert c.err.item() == 0
    L = c.L
    logits, idx, w, out = definition(L, u, c.K, executed)
    tau = logit_tau(L, u)
    assert ((c.logits.double() - logits).abs().cpu().numpy() <= tau).all()
    check_topk(c.idx.cpu().numpy(), logits.cpu().numpy(), tau, c.K)
    if executed is None and not torch.equal(c.idx.long(), idx):  # a near tie that the rule above allows
        logits, idx, w, out = definition(L, u, c.K, c.idx)
    # softmax over logits that are off by tau: at most 2 tau relative, and the fp32 steps
    assert ((c.w.double() - w).abs().cpu().numpy() <= (2 * tau.max(1)[:, None] + 32 * EPS32) * w.cpu().numpy()).all()
    wtol = 2 * float(tau.max())
    got = c.out.double() if base is None else c.out.double() - base.double()
    tol = OUT_TOL + min(wtol, 1e-5)
    if c.mode == M.OUT_BF16:
        tol += EPSBF
    if base is not None:  # the sum's rounding, relative to the sum
        tol += EPS32 * (c.out.double().norm(dim=1) / out.norm(dim=1)).max().item()
    assert rel(got, out) <= tol, (rel(got, out), tol)
    lo = c.out.data_ptr() - c.buf.data_ptr()
    n = lo // c.buf.element_size()
    if 0 <= n <= 64:
        assert (c.buf[:n] == 7).all() and (c.buf[n + c.T * L.H:] == 7).all()


def tokens(T, H, seed=0, spread=True):
    g = torch.Generator(device=DEV).manual_seed(seed * 131 + T + H)
    x = torch.randn((T, H), device=DEV, generator=g)
    return x * (torch.rand((T, 1), device=DEV, generator=g) * 3 + 0.2) if spread else x


# ----------------------------------------------------------------------------- shapes and types
@pytest.mark.parametrize("T,H,E,K,I,r", [
    (1, 256, 16, 2, 128, 8), (4, 256, 16, 2, 128, 8), (2, 256, 1, 1, 128, 0), (32, 256, 5, 5, 128, 16), (3, 512, 256, 8, 256, 24),
    (1, 2048, 256, 4, 512, 16), (5, 2048, 128, 8, 512, 16), (16, 2048, 256, 4, 512, 0), (17, 2048, 33, 3, 512, 32),
    (32, 2048, 64, 8, 512, 16), (7, 4096, 20, 4, 1024, 16), (9, 4096, 12, 2, 128, 0), (32, 4096, 9, 8, 256, 8),
    (6, 256, 40, 6, 2048, 16), (13, 1024, 77, 7, 1024, 8), (1, 4096, 8, 8, 2048, 32)])
def test_layer(cuda_ok, T, H, E, K, I, r):
    L = Layer(H, E, I, r)
    x = tokens(T, H)
    c = Call(L, T, K)
    u_out = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    c(u=u_out, x=x)
    u = normed(x)
    check(c, u)
    assert torch.equal(u_out, u)
    c2 = Call(L, T, K, M.OUT_BF16, offset=1)  # an output that is aligned to its elements only
    c2(u=u.contiguous())
    check(c2, u)


@pytest.mark.parametrize("T", [1, 6, 20])
@pytest.mark.parametrize("sh,down,gate_up", [((True, False, False), False, False), ((False, True, True), True, False),
                                             ((False, False, True), False, True), ((False, False, False), True, True),
                                             ((True, True, True), True, True)])
def test_adapters_each_alone_and_together(cuda_ok, T, sh, down, gate_up):
    L = Layer(512, 24, 256, 24, sh, down, gate_up, lora_scale=0.75)
    x = tokens(T, 512)
    c = Call(L, T, 4)(x=x)
    check(c, normed(x))


@pytest.mark.parametrize("T,K", [(1, 1), (9, 4), (32, 8)])
def test_given_experts(cuda_ok, T, K):
    """exec_idx: any experts, one listed twice, ids outside clamped; idx stays the router's own top-K."""
    L = Layer(512, 20, 256, 16, down=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    ex = torch.randint(0, 20, (T, K), dtype=torch.int32, device=DEV, generator=g)
    ex[0, 0] = -7
    ex[-1, -1] = 1000
    if K > 1:
        ex[0, 1] = ex[0, 0]
    u = tokens(T, 512, spread=False).bfloat16()
    c = Call(L, T, K)(u=u, executed=ex)
    check(c, u, ex)


def test_every_token_on_the_same_experts(cuda_ok):
    """32 tokens in one bucket: more slots of an expert than one pass takes."""
    L = Layer(512, 30, 256, 8, down=True, gate_up=True)
    L.bias[3], L.bias[29] = 1000.0, 990.0
    u = tokens(32, 512).bfloat16()
    c = Call(L, 32, 2)(u=u)
    check(c, u)
    assert (c.idx == torch.tensor([3, 29], dtype=torch.int32, device=DEV)).all()


@pytest.mark.parametrize("T", [2, 12])
def test_residual_in_place(cuda_ok, T):
    L = Layer(512, 24, 256, 16)
    x = tokens(T, 512)
    u, base = normed(x), x.clone()
    c = Call(L, T, 4, M.OUT_ADD_F32)
    c(x=x, out=x, logits=True)
    c.out = x
    check(c, u, base=base)


def test_no_logits_and_no_tokens(cuda_ok):
    L = Layer(256, 16, 128, 8)
    u = tokens(3, 256).bfloat16()
    c, d = Call(L, 3, 2)(u=u), Call(L, 3, 2)(u=u, logits=False)
    torch.cuda.synchronize()
    assert torch.equal(c.out, d.out) and torch.equal(c.idx, d.idx) and torch.equal(c.w, d.w)
    M.moe_layer_decode(L.dev, u[:0], 2, c.idx, c.w, c.out, 0, c.ws)


def test_layer_said_to_be_elsewhere(cuda_ok):
    L = Layer(256, 16, 128, 0)
    c = Call(L, 3, 2)
    L.dev.device = torch.device("cuda", torch.cuda.current_device() + 1)
    with pytest.raises(ValueError, match="the layer is on"):
        c(u=tokens(3, 256).bfloat16())
    torch.cuda.synchronize()
    assert (c.idx == -1).all() and (c.buf == 7).all()


# ----------------------------------------------------------------------------- values
@pytest.mark.parametrize("mag", [1e-36, 1e-8, 3.0, 1e3])
def test_magnitudes_of_u(cuda_ok, mag):
    """bf16 tokens of any size, entries of one token spread over 12 binary orders; a zero row beside them."""
    L = Layer(512, 16, 128, 8, scale=min(1.0, 1 / mag))
    T = 5
    g = torch.Generator(device=DEV).manual_seed(3)
    u = (tokens(T, 512) * mag * 2.0 ** -torch.randint(0, 13, (T, 512), device=DEV, generator=g)).bfloat16()
    u[2] = 0
    c = Call(L, T, 3)(u=u)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    logits, idx, w, out = definition(L, u, 3, c.idx)
    assert ((c.logits.double() - logits).abs().cpu().numpy() <= logit_tau(L, u)).all()
    rows = [0, 1, 3, 4]
    if mag > 1e-30:  # below, the hidden values fall under fp16's smallest steps and the outputs are zero to fp32
        n = out[rows].norm(dim=1)
        floor = 0 if mag > 1e-3 else 1.0  # h below 2^-14 keeps 2^-36 absolutely
        if not floor:
            assert rel(c.out[rows], out[rows]) <= OUT_TOL + 1e-5
        else:
            # 2^-36 per hidden value through I weights of at most 0.5, K + 1 experts
            assert ((c.out[rows].double() - out[rows]).norm(dim=1) <= OUT_TOL * n + 4 * 2.0 ** -36 * 128 * 512 ** 0.5).all()
    assert (c.out[2] == 0).all()


@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("mag,share", [(1e-2, 1e-6), (1e-3, 1e-4), (1e-4, 1e-2)])
def test_small_tokens_keep_what_the_header_says(cuda_ok, mag, share, down):
    """Hidden values under 2^-14 are rounded by at most 2^-36 each: a vector of I of them by sqrt(I) 2^-36, which the down
    projection (with its adapter) stretches by its largest singular value at most; the K experts' weights add up to 1, the
    shared expert's gate is at most 1.  `share` of the output bounds all of it, so an output that is lost fails."""
    H, I, K, T = 512, 128, 3, 5
    L = Layer(H, 16, I, 8, down=down)
    u = (tokens(T, H, spread=False) * mag).bfloat16()
    c = Call(L, T, K)(u=u)
    torch.cuda.synchronize()
    assert c.err.item() == 0
    out = definition(L, u, K, c.idx)[3]
    cut = 2 * I * M.qrow_bytes(H, 4)

    def stretch(block, p):
        D = matrix(block[cut:cut + H * M.qrow_bytes(I, 4)].view(H, -1), I, 4)
        if p is not None:
            D = D + p[1].double() @ p[0].double()
        return torch.linalg.matrix_norm(D, 2).item()

    most = max(stretch(L.pool[e], (L.down[0][e], L.down[1][e]) if down else None) for e in range(16))
    floor = (most + stretch(L.shared, L.sh[2])) * I ** 0.5 * 2.0 ** -36
    n = out.norm(dim=1)
    assert (floor <= share * n).all()
    assert ((c.out.double() - out).norm(dim=1) <= (OUT_TOL + 1e-5) * n + floor).all()


def test_non_finite_tokens_stay_alone(cuda_ok):
    """NaN and infinite entries make their own token NaN; ids stay in range; the others are as without them."""
    L = Layer(512, 16, 128, 8, down=True, gate_up=True)
    for T in (4, 31):
        for with_x in (False, True):
            x = tokens(T, 512)
            clean = Call(L, T, 3)
            bad = Call(L, T, 3)
            y = x.clone()
            y[1, 5], y[2, 7] = float("nan"), float("inf")
            if with_x:
                clean(x=x), bad(x=y)
            else:
                clean(u=x.bfloat16()), bad(u=y.bfloat16())
            torch.cuda.synchronize()
            assert ((bad.idx >= 0) & (bad.idx < 16)).all()
            assert all(len(set(r)) == 3 for r in bad.idx.tolist())
            assert torch.isnan(bad.out[1]).any() and not torch.isfinite(bad.out[2]).all()
            keep = [t for t in range(T) if t not in (1, 2)]
            assert torch.equal(bad.out[keep], clean.out[keep]) and torch.equal(bad.idx[keep], clean.idx[keep])


def test_hidden_values_beyond_fp16_are_reported(cuda_ok):
    L = Layer(256, 16, 128, 0, scale=30.0)
    u = (tokens(2, 256) * 40).bfloat16()
    c = Call(L, 2, 2)(u=u)
    torch.cuda.synchronize()
    assert c.err.item() == _lib.MOE_ERR_RANGE


def test_equal_logits_go_to_the_lower_expert(cuda_ok):
    L = Layer(256, 40, 128, 0, bias=0.0)
    L.router[:] = L.router[:1]
    u = tokens(3, 256).bfloat16()
    c = Call(L, 3, 8)(u=u)
    torch.cuda.synchronize()
    assert (c.idx == torch.arange(8, device=DEV)).all() and ((c.w - 0.125).abs() < 1e-6).all()


# ----------------------------------------------------------------------------- streams, graphs, neighbours
def test_repeats_streams_and_graphs(cuda_ok):
    """The same call again, with its workspace full of something else, on another stream and replayed from a graph."""
    L = Layer(512, 24, 256, 16, down=True)
    for T in (1, 9):
        x = tokens(T, 512)
        c = Call(L, T, 4)(x=x)
        torch.cuda.synchronize()
        first = c.out.clone()
        for fill in (0, 0xFF, 0x01):
            c.ws.fill_(fill)
            c(x=x)
            c(x=x)
            torch.cuda.synchronize()
            assert torch.equal(c.out, first)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            c(x=x)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(c.out, first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c(x=x)
        c.ws.fill_(0x5A)
        for _ in range(3):
            c.out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.out, first)
        assert c.err.item() == 0


@pytest.mark.parametrize("T", [2, 9])
def test_workspace_written_to_in_part(cuda_ok, T):
    """Any four bytes of what a call leaves at the head of its workspace written over: the next call is as the first."""
    L = Layer(512, 24, 256, 16, down=True)
    x = tokens(T, 512)
    c = Call(L, T, 4)(x=x)
    torch.cuda.synchronize()
    first = c.out.clone()
    words = c.ws[:64].view(torch.int32)
    for i in range(16):
        for v in (0, 1, 148, -1, 0x10000):
            words[i] = v
            c.out.zero_()
            c(x=x)
            torch.cuda.synchronize()
            assert torch.equal(c.out, first) and c.err.item() == 0, (i, v)
    words.zero_()
    c(x=x)
    torch.cuda.synchronize()
    assert torch.equal(c.out, first) and c.err.item() == 0


@pytest.mark.parametrize("late", [0, 1, 147])
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("T,routed", [(2, False), (2, True), (9, True)])
def test_waits_that_run_out(cuda_ok, T, routed, fresh, late):
    """One CTA four limits late: the others' waits (at a barrier, or for CTA 0 to set a fresh workspace's counters up) run
    out and say so, the call ends, and the next ones on the same workspace are as if it had not been."""
    H, K = 512, 4
    layers = [Layer(H, 24, 256, 16, down=routed, gate_up=routed, seed=s) for s in range(2)]
    st = M.StackStructs([l.dev for l in layers])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = M.workspace(M.moe_stack_workspace_size(st, T, K, K))
    x0 = tokens(T, H)

    def run(**kw):
        x = x0.clone()
        M.moe_stack_decode(st, x, K, K, EPS, ws, err_word=err, opts=M.stack_opts(path=M.PATH_LAYER_DECODE, **kw))
        torch.cuda.synchronize()
        return x, err.item()

    good, code = run()
    assert code == 0
    for layer in (0, 1, 0):
        if fresh:
            ws.fill_(0xA5)
        assert run(timeout_ns=2_000_000, drop_layer=layer, drop_cta=late)[1] == _lib.MOE_ERR_TIMEOUT
        for _ in range(3):
            x, code = run()
            assert code == 0 and torch.equal(x, good)


def test_two_calls_at_once(cuda_ok):
    """Two streams, each with its own workspace, many calls in flight."""
    L = Layer(512, 24, 256, 16)
    a, b = Call(L, 2, 4), Call(L, 11, 4)
    xa, xb = tokens(2, 512), tokens(11, 512)
    a(x=xa), b(x=xb)
    torch.cuda.synchronize()
    ra, rb = a.out.clone(), b.out.clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(50):
        with torch.cuda.stream(s1):
            a(x=xa)
        with torch.cuda.stream(s2):
            b(x=xb)
    torch.cuda.synchronize()
    assert torch.equal(a.out, ra) and torch.equal(b.out, rb) and a.err.item() == b.err.item() == 0


def test_beside_products_on_another_stream(cuda_ok):
    """The layer on one stream, quantiser and product (rows, cluster split, CTA pairs) on another, many calls in flight:
    each is as it is alone."""
    L = Layer(512, 24, 256, 16, down=True)
    a = Call(L, 11, 4)
    xa = tokens(11, 512)
    a(x=xa)
    g = torch.Generator(device=DEV).manual_seed(2)
    work = []
    for N, H, T in ((4096, 2048, 1), (2048, 1024, 40), (8192, 512, 300)):
        lin = M.DeviceLinear8(torch.randint(-128, 128, (N, H), dtype=torch.int8, device=DEV, generator=g),
                              torch.rand(N, device=DEV, generator=g))
        work.append((lin, torch.randn((T, H), device=DEV, generator=g), torch.empty((T, H), dtype=torch.int8, device=DEV),
                     torch.empty(T, device=DEV), torch.empty((T, N), device=DEV)))

    def products():
        for lin, x, q, s, out in work:
            M.moe_quant_i8(x, q, s, eps=EPS)
            M.moe_linear_i8(lin, q, s, out, M.OUT_F32)

    products()
    torch.cuda.synchronize()
    want, outs = a.out.clone(), [w[-1].clone() for w in work]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(60):
        with torch.cuda.stream(s1):
            a(x=xa)
        with torch.cuda.stream(s2):
            products()
    torch.cuda.synchronize()
    assert torch.equal(a.out, want) and a.err.item() == 0
    assert all(torch.equal(w[-1], o) for w, o in zip(work, outs))


def test_agrees_with_route_and_expert_forward(cuda_ok):
    """The library's separate calls on the same layer: the same experts, outputs within their stated tolerance."""
    L = Layer(2048, 64, 512, 16)
    for T in (3, 24):
        u = tokens(T, 2048, spread=False).bfloat16()
        c = Call(L, T, 4)(u=u)
        logits, idx, w = torch.empty((T, 64), device=DEV), torch.empty_like(c.idx), torch.empty_like(c.w)
        M.moe_route_topk(L.dev, u, 4, logits, idx, w)
        out = torch.empty((T, 2048), device=DEV)
        M.moe_expert_forward(L.dev, u, 4, idx, w, out, M.OUT_F32, M.workspace(M.moe_workspace_size(L.dev, T, 4)))
        torch.cuda.synchronize()
        assert torch.equal(idx, c.idx) and torch.allclose(w, c.w, rtol=1e-4)
        assert (out - c.out).abs().max() <= 2e-3 * out.abs().max()


@pytest.mark.parametrize("T", [1, 7])
def test_projection_then_layer(cuda_ok, T):
    """The calls as a decoder makes them: x += projection of rmsnorm(x) in 8 bits, then x += layer(x), twice over,
    captured in one graph; against 64 bits step by step."""
    H = 512
    L = Layer(H, 24, 256, 16)
    g = torch.Generator(device=DEV).manual_seed(9)
    W = torch.randint(-127, 128, (H, H), dtype=torch.int8, device=DEV, generator=g)
    sw = torch.rand(H, device=DEV, generator=g) * 1e-3
    lin = M.DeviceLinear8(W, sw)
    x0 = tokens(T, H)
    x, q, s = x0.clone(), torch.zeros((T, H), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    c = Call(L, T, 4, M.OUT_ADD_F32)
    mids = [torch.empty_like(x) for _ in range(4)]

    def step():
        for i in range(2):
            M.moe_quant_i8(x, q, s, eps=EPS)
            M.moe_linear_i8(lin, q, s, x, M.OUT_ADD_F32)
            mids[2 * i].copy_(x)
            c(x=x, out=x)
            mids[2 * i + 1].copy_(x)

    step()
    torch.cuda.synchronize()
    x.copy_(x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(x0)
    graph.replay()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    before = x0
    for i in range(2):
        d = before.double()
        m = d.abs().amax(1, keepdim=True)
        unit = m / (d.square().mean(1, keepdim=True) + EPS).sqrt() / 127
        y = ((127 * d / m).round() @ W.double().T) * unit * sw.double()
        assert rel(mids[2 * i], d + y) <= 16 * EPS32  # 14 roundings of the scale and the product, one of the sum
        after = mids[2 * i]
        out = definition(L, normed(after), 4)[3]
        assert rel(mids[2 * i + 1], after.double() + out) <= OUT_TOL + 1e-5
        before = mids[2 * i + 1]


# ----------------------------------------------------------------------------- as a path of the stack
@pytest.mark.parametrize("T,predicted", [(1, False), (3, True), (9, False), (32, True)])
def test_stack_path(cuda_ok, T, predicted):
    """moe_stack_decode with one launch a layer: every layer's step from the traces, against 64 bits; the Prerouter's
    predictions as the per-layer path makes them."""
    H, E, I, K, P = 512, 24, 256, 4, 64
    layers = [Layer(H, E, I, 16, down=True, seed=s) for s in range(3)]
    g = torch.Generator(device=DEV).manual_seed(11)

    class Head:
        def __init__(self):
            self.t = {n: (torch.randn(sh, device=DEV, generator=g) / sh[-1] ** 0.5).half()
                      for n, sh in (("W1", (P, H + E)), ("b1", (P,)), ("W2", (E, P)), ("b2", (E,)))}
            self.struct = _lib.moe_prerouter(*(self.t[n].data_ptr() for n in ("W1", "b1", "W2", "b2")), H, E, P, E)

    heads = [Head() for _ in layers]
    st = M.StackStructs([l.dev for l in layers], heads)
    n = len(layers)

    def run(path):
        x = tokens(T, H)
        o = dict(x_trace=torch.zeros((n, T, H), device=DEV), u_trace=torch.zeros((n, T, H), dtype=torch.bfloat16, device=DEV),
                 idx_all=torch.zeros((n, T, K), dtype=torch.int32, device=DEV),
                 true_idx_all=torch.zeros((n, T, K), dtype=torch.int32, device=DEV),
                 pred_all=torch.zeros((n, T, K), dtype=torch.int32, device=DEV))
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = M.workspace(M.moe_stack_workspace_size(st, T, K, K))
        ws.fill_(0xC3)
        M.moe_stack_decode(st, x, K, K, EPS, ws, use_predicted_routing=predicted, err_word=err,
                           opts=M.stack_opts(path=path), **o)
        torch.cuda.synchronize()
        assert err.item() == 0
        return x, o

    x, o = run(M.PATH_LAYER_DECODE)
    _, ref = run(M.PATH_LAYERS)
    assert torch.equal(o["u_trace"][0], ref["u_trace"][0]) and torch.equal(o["true_idx_all"][0], ref["true_idx_all"][0])
    assert torch.equal(o["pred_all"][0], ref["pred_all"][0])
    for l, L in enumerate(layers):
        before, after = o["x_trace"][l], o["x_trace"][l + 1] if l + 1 < n else x
        u = o["u_trace"][l]
        assert torch.equal(u, normed(before))
        ex = o["pred_all"][l - 1] if predicted and l else o["true_idx_all"][l]
        assert torch.equal(o["idx_all"][l], ex)
        out = definition(L, u, K, ex)[3]
        # the layer's tolerance, and the sum's rounding relative to the sum
        tol = OUT_TOL + 1e-5 + EPS32 * (after.double().norm(dim=1) / out.norm(dim=1)).max().item()
        assert rel(after.double() - before.double(), out) <= tol


@pytest.mark.parametrize("path", [M.PATH_LAYERS, M.PATH_LAYER_DECODE])
@pytest.mark.parametrize("T", [1, 9])
def test_stack_with_adapters_on_later_layers_only(cuda_ok, T, path):
    """Layers share the shapes and not the adapters: one without routed adapters, one with them on the down projections,
    one on gate and up too; a workspace of exactly the size that the query names."""
    H, E, I, K = 512, 24, 256, 4
    layers = [Layer(H, E, I, 16, seed=0), Layer(H, E, I, 16, down=True, seed=1),
              Layer(H, E, I, 16, down=True, gate_up=True, seed=2)]
    st = M.StackStructs([l.dev for l in layers])
    x = tokens(T, H)
    traces, u = torch.zeros((3, T, H), device=DEV), torch.zeros((3, T, H), dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros((3, T, K), dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = M.workspace(M.moe_stack_workspace_size(st, T, K, K))
    M.moe_stack_decode(st, x, K, K, EPS, ws, x_trace=traces, u_trace=u, idx_all=idx, err_word=err,
                       opts=M.stack_opts(path=path))
    torch.cuda.synchronize()
    assert err.item() == 0
    for l, L in enumerate(layers):
        before, after = traces[l], traces[l + 1] if l + 1 < 3 else x
        out = definition(L, u[l], K, idx[l])[3]
        # the per-layer path multiplies fp16 operands, rounded weights and hidden values among them (2^-11 each)
        tol = OUT_TOL + 1e-5 if path == M.PATH_LAYER_DECODE else 2e-3
        tol += EPS32 * (after.double().norm(dim=1) / out.norm(dim=1)).max().item()
        assert rel(after.double() - before.double(), out) <= tol


def test_stack_path_refuses_many_tokens(cuda_ok):
    L = Layer(256, 16, 128, 8)
    st = M.StackStructs([L.dev])
    x = torch.zeros((33, 256), device=DEV)
    with pytest.raises(M.MoEError) as e:
        M.moe_stack_decode(st, x, 2, 2, EPS, M.workspace(M.moe_stack_workspace_size(st, 33, 2, 2)),
                           opts=M.stack_opts(path=M.PATH_LAYER_DECODE))
    assert e.value.code == _lib.MOE_ERR_UNSUPPORTED
