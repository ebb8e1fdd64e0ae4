"""GPU parity of the 8-bit product and its quantiser against integer and 64-bit definitions.

Codes are compared exactly with the correctly rounded quotient (rational arithmetic where 64 bits tie), integer sums
are exact, so the only allowance is for the fp32 steps around them: EPS32 each.
"""
import numpy as np
import pytest
import torch

import int4_expert_ffn_top_b200 as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS32 = torch.finfo(torch.float32).eps / 2
EPSBF = torch.finfo(torch.bfloat16).eps / 2


def codes_of(x):
    """round_half_even(127 x / max|x|) per row, in 64 bits: 127 x is exact there, and a quotient of two fp32 values
    that is not a tie is further from one than a double's rounding."""
    x = x.double()
    m = x.abs().amax(1, keepdim=True)
    return torch.where(m > 0, (127 * x / torch.where(m > 0, m, torch.ones_like(m))).round(), torch.zeros_like(x)), m[:, 0]


def quant(x, eps=None, pad=0, fill=77):
    T, H = x.shape
    ld = M.moe_i8_row_bytes(H) + 16 * pad
    q = torch.full((T, ld), fill, dtype=torch.int8, device=DEV)
    s = torch.full((T,), float("nan"), device=DEV)
    M.moe_quant_i8(x, q, s, eps=eps)
    torch.cuda.synchronize()
    assert (q[:, H:] == fill).all()  # bytes past the row stay
    return q, s


def linear(N, K, seed=0, bias=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    W = torch.randint(-128, 128, (N, K), dtype=torch.int8, device=DEV, generator=g)
    sw = torch.rand(N, device=DEV, generator=g) * 0.01 + 1e-4
    b = torch.randn(N, device=DEV, generator=g) if bias else None
    return M.DeviceLinear8(W, sw, b), W, sw, b


def product64(W, sw, b, q, sx, K):
    p = (q[:, :K].double() @ W.double().T) * sx.double()[:, None] * sw.double()
    return p, p if b is None else p + b.double()


def check_linear(N, K, T, mode, bias=True, pad=0, seed=0):
    lin, W, sw, b = linear(N, K, seed, bias)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    q = torch.randint(-128, 128, (T, M.moe_i8_row_bytes(K) + 16 * pad), dtype=torch.int8, device=DEV, generator=g)
    sx = torch.rand(T, device=DEV, generator=g) * 0.1
    tail = 64
    out = torch.full((T * N + tail,), 3.0, device=DEV, dtype=torch.bfloat16 if mode == M.OUT_BF16 else torch.float32)
    if mode == M.OUT_ADD_F32:
        out[:T * N] = torch.randn(T * N, device=DEV, generator=g)
    before = out.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    M.moe_linear_i8(lin, q, sx, out, mode, err_word=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    p, ref = product64(W, sw, b, q, sx, K)
    # int -> fp32, two scales, the bias: one rounding each
    tol = 3.01 * EPS32 * p.abs() + 1.01 * EPS32 * ref.abs()
    if mode == M.OUT_BF16:
        tol = tol + 1.01 * EPSBF * ref.abs()
    elif mode == M.OUT_ADD_F32:
        ref = ref + before[:T * N].view(T, N).double()
        tol = tol + 1.01 * EPS32 * ref.abs()
    off = (out[:T * N].view(T, N).double() - ref).abs() - tol
    assert off.max().item() <= 0, off.max().item()
    assert torch.equal(out[T * N:], before[T * N:])  # nothing written behind the last row


# ----------------------------------------------------------------------------- quantiser
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 17), (5, 2048), (2, 1000), (7, 255), (1, 65536), (300, 4096), (2, 9999),
                                 (1184, 2048), (1190, 264), (1185, 257)])
def test_codes_are_the_correctly_rounded_quotients(cuda_ok, T, H, dtype):
    g = torch.Generator(device=DEV).manual_seed(T * H)
    x = (torch.randn((T, H), device=DEV, generator=g) * torch.rand((T, 1), device=DEV, generator=g).add(0.1)).to(dtype)
    for eps in (None, 1e-6):
        q, s = quant(x, eps, pad=T % 2)
        ref, m = codes_of(x)
        assert torch.equal(q[:, :H].double(), ref)
        if eps is not None:
            m = m / (x.double().square().mean(1) + eps).sqrt()
        # the sum of squares: H/256 terms a thread, 5 + 8 joining steps, each one rounding, halved by the root;
        # then mean, eps, root, reciprocal, product and /127
        tol = (0.5 * (H / 256 + 16) + 6 if eps is not None else 1) * 1.01 * EPS32
        assert ((s.double() * 127 / m) - 1).abs().max().item() <= tol


def test_codes_at_ties_and_next_to_them(cuda_ok):
    """m = 254 puts x = n + 1/2 steps exactly between two codes at odd integers; its neighbours lie to either side."""
    n = torch.arange(-253, 254, 2, dtype=torch.float32)
    x = torch.cat([n, torch.nextafter(n, n + 1), torch.nextafter(n, n - 1), torch.tensor([254.0, -254.0])])[None]
    q, _ = quant(x.to(DEV))
    h = (x[0].numpy().astype(np.float64) / 2)
    assert np.array_equal(q[0, :x.shape[1]].cpu().numpy(), np.rint(h).astype(np.int8))
    assert np.array_equal(np.rint(h[:254]) % 2, np.zeros(254))  # the ties go to even codes


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e30, 3e38])
def test_extreme_magnitudes(cuda_ok, scale):
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.rand((4, 100), device=DEV, generator=g) * 2 - 1) * scale
    q, s = quant(x)
    ref, m = codes_of(x)
    assert torch.equal(q[:, :100].double(), ref)
    assert ((s.double() - m / 127).abs() <= EPS32 * 1.01 * m / 127 + 2.0 ** -150).all()


@pytest.mark.parametrize("H", [104, 2000, 65536])
@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-25, 1e-16, 1e15, 1e17, 1e20, 1e30, 3e38])
def test_norm_of_extreme_magnitudes(cuda_ok, scale, H):
    """Rows whose squares overflow or vanish in fp32: the scale still holds."""
    g = torch.Generator(device=DEV).manual_seed(H)
    for dtype in (torch.float32, torch.bfloat16):
        x = ((torch.rand((3, H), device=DEV, generator=g) * 2 - 1) * scale).to(dtype)
        for eps in (0.0, 1e-6):
            q, s = quant(x, eps)
            ref, m = codes_of(x)
            assert torch.equal(q[:, :H].double(), ref)
            want = torch.where(m > 0, m / (x.double().square().mean(1) + eps).sqrt() / 127, 0.0)
            tol = (0.5 * (H / 256 + 16) + 6) * 1.01 * EPS32
            assert ((s.double() - want).abs() <= tol * want + 2.0 ** -149).all()


def test_zero_and_non_finite_rows(cuda_ok):
    x = torch.randn((6, 70), device=DEV)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 69] = float("inf")
    x[3, 0] = float("-inf")
    x[4, 5], x[4, 6] = float("nan"), float("inf")
    for eps in (None, 0.0):
        q, s = quant(x, eps)
        assert (q[:5, :70] == 0).all() and s[0].item() == 0 and torch.isnan(s[1:5]).all() and torch.isfinite(s[5])
        assert torch.equal(q[5:, :70].double(), codes_of(x[5:])[0])


# ----------------------------------------------------------------------------- product
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("N,K,T", [(1, 1, 1), (16, 64, 1), (17, 63, 3), (2051, 1000, 13), (4096, 2048, 1), (33, 65, 8),
                                   (100, 4096, 9), (257, 129, 16), (48, 333, 31), (640, 2048, 64), (300, 144, 65),
                                   (129, 255, 127), (256, 512, 128), (513, 1040, 300), (2048, 2048, 256)])
def test_product(cuda_ok, N, K, T, mode):
    check_linear(N, K, T, mode, bias=(N + T) % 2 == 0, pad=T % 3, seed=N + T)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("N,K,T", [
    (9000, 3000, 2), (9000, 40, 4), (5000, 100, 5), (70000, 64, 7),  # few tokens, many rows: no split of K, and little K
    (200000, 512, 1), (131072, 1000, 2), (4096, 2048, 3), (2051, 1008, 8),  # both sides of the few-token rule
    (30000, 333, 16), (40000, 144, 20), (65536, 100, 32),  # more tiles of 32 tokens than multiprocessors
    (20001, 272, 50), (70000, 130, 33), (80001, 64, 20),  # CTA pairs, 64 tokens a tile, several tiles a pair
    (4100, 1000, 450), (4099, 2050, 600), (4100, 144, 1000),  # 128, 192 and 256 tokens a tile, ragged last tiles
    (4353, 130, 1025), (9001, 300, 2000), (4097, 4111, 513)])
def test_product_of_many_tiles(cuda_ok, N, K, T, mode):
    check_linear(N, K, T, mode, bias=(N + T) % 2 == 0, pad=T % 3, seed=N + T)


@pytest.mark.parametrize("T", [1, 70, 130])
def test_largest_sum_is_exact(cuda_ok, T):
    """All codes -128 over the longest rows: the largest magnitude a 32-bit sum has to hold."""
    K, N = 65536, 20
    lin = M.DeviceLinear8(torch.full((N, K), -128, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
    q = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
    out = torch.empty((T, N), device=DEV)
    M.moe_linear_i8(lin, q, torch.ones(T, device=DEV), out, M.OUT_F32)
    assert (out == float(128 * 128 * K)).all()


def test_non_finite_scales_stay_in_their_rows(cuda_ok):
    lin, W, sw, b = linear(40, 64)
    for T in (3, 130):
        q = torch.ones((T, 64), dtype=torch.int8, device=DEV)
        sx = torch.ones(T, device=DEV)
        sx[1] = float("nan")
        out = torch.empty((T, 40), device=DEV)
        M.moe_linear_i8(lin, q, sx, out, M.OUT_F32)
        assert torch.isnan(out[1]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[2:]).all()


@pytest.mark.parametrize("T", [1, 40, 200])
def test_quantised_projection_as_used(cuda_ok, T):
    """Residual stream -> normed codes -> product added to the residual, against 64 bits, eagerly on another stream
    and replayed from a graph."""
    H, N = 512, 512
    lin, W, sw, _ = linear(N, H, bias=False)
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, H), device=DEV, generator=g)
    q = torch.zeros((T, H), dtype=torch.int8, device=DEV)
    s = torch.empty(T, device=DEV)
    out = x.clone()

    def call():
        M.moe_quant_i8(x, q, s, eps=1e-6)
        M.moe_linear_i8(lin, q, s, out, M.OUT_ADD_F32)

    ref, m = codes_of(x)
    unit = m / (x.double().square().mean(1) + 1e-6).sqrt() / 127
    p = (ref @ W.double().T) * unit[:, None] * sw.double()
    # the scale's roundings (see above) and the product's
    tol = ((0.5 * (H / 256 + 16) + 6) + 3) * 1.01 * EPS32 * p.abs() + 1.01 * EPS32 * (p + x.double()).abs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert ((out.double() - x.double() - p).abs() <= tol).all()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.copy_(x)
    q.fill_(5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("N,K,T", [
    (4096, 2048, 1), (8192, 4096, 2), (1024, 1024, 4), (512, 512, 8),  # dp4a rows
    (4096, 2048, 8), (2048, 2048, 64), (30000, 512, 16),  # K split over a cluster
    (8192, 2048, 200), (4100, 4096, 600)])  # CTA pairs
def test_matrix_that_the_quantiser_has_just_written(cuda_ok, N, K, T):
    """The call right before the product writes the matrix's codes and scales, over those of another matrix: none of the
    old ones may reach the product, eagerly or from a graph."""
    g = torch.Generator(device=DEV).manual_seed(N + K + T)
    x = torch.randn((T, K), device=DEV, generator=g)
    q, sx = torch.empty((T, K), dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    codes, sw = torch.zeros((N, K), dtype=torch.int8, device=DEV), torch.zeros(N, device=DEV)
    lin = M.DeviceLinear8(codes, sw)
    assert lin.codes.data_ptr() == codes.data_ptr()
    Wf, out = torch.empty((N, K), device=DEV), torch.empty((T, N), device=DEV)

    def call():
        M.moe_quant_i8(x, q, sx)
        M.moe_quant_i8(Wf, codes, sw)
        M.moe_linear_i8(lin, q, sx, out, M.OUT_F32)

    Wf.normal_(generator=g)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(12):
        Wf.normal_(generator=g)
        call() if i % 2 else graph.replay()
        torch.cuda.synchronize()
        first = out.clone()
        assert torch.equal(codes.double(), codes_of(Wf)[0])
        p, ref = product64(codes, sw, None, q, sx, K)
        assert ((first.double() - ref).abs() <= 3.01 * EPS32 * p.abs()).all()


def test_call_that_waits_for_room_in_the_queue(cuda_ok):
    """More calls than the device's queue holds, from two threads on their own streams: each waits without the
    interpreter's lock, and both results hold."""
    import threading
    lin, W, sw, b = linear(512, 512, seed=3)
    outs = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            g = torch.Generator(device=DEV).manual_seed(k)
            x = torch.randn((64, 512), device=DEV, generator=g)
            q = torch.zeros((64, 512), dtype=torch.int8, device=DEV)
            s = torch.empty(64, device=DEV)
            out = torch.empty((64, 512), device=DEV)
            for _ in range(1500):
                M.moe_quant_i8(x, q, s)
                M.moe_linear_i8(lin, q, s, out, M.OUT_F32)
            torch.cuda.current_stream().synchronize()
            outs.append((q, s, out))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert len(outs) == 2
    for q, s, out in outs:
        p, ref = product64(W, sw, b, q, s, 512)
        assert ((out.double() - ref).abs() <= 3.01 * EPS32 * p.abs() + 1.01 * EPS32 * ref.abs()).all()


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    """The product's kernels with a limit of the test's (linear8_waits.cu)."""
    import ctypes
    import os
    import subprocess

    from int4_expert_ffn_top_b200 import _lib, build

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = str(tmp_path_factory.mktemp("waits") / "linear8_waits.so")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "linear8_waits.cu")
    subprocess.run([build.nvcc(), *build.NVCC_FLAGS, "-Xlinker", "-Bsymbolic", "-o", lib, src], check=True)
    fn = ctypes.CDLL(lib).linear8_waits
    c = ctypes
    fn.argtypes = [c.c_int, c.POINTER(_lib.moe_linear8), c.c_void_p, c.c_int64, c.c_void_p, c.c_int32, c.c_void_p, c.c_void_p,
                   c.c_int64, c.c_int, c.c_void_p]
    return fn


@pytest.mark.parametrize("kind,starve,N,K,T", [(0, 1, 700, 300, 100), (0, 1, 20001, 2048, 200), (0, 1, 256, 4096, 64),
                                               (1, 1, 700, 300, 30), (1, 2, 700, 2048, 30), (1, 1, 300, 2048, 90)])
def test_waits_that_run_out(cuda_ok, waits, kind, starve, N, K, T):
    """Operands that never become complete: the calls end, say so, and leave the multiprocessors as they were (tensor
    memory, barriers) for the products after them."""
    import ctypes

    from int4_expert_ffn_top_b200 import _lib
    lin, W, sw, b = linear(N, K, seed=4)
    g = torch.Generator(device=DEV).manual_seed(4)
    ld = M.moe_i8_row_bytes(K)
    q = torch.randint(-128, 128, (T, ld), dtype=torch.int8, device=DEV, generator=g)
    sx = torch.rand(T, device=DEV, generator=g) * 0.1
    out, err = torch.empty((T, N), device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    p, ref = product64(W, sw, b, q, sx, K)
    tol = 3.01 * EPS32 * p.abs() + 1.01 * EPS32 * ref.abs()

    def call(limit_ns, starved):
        err.zero_()
        out.fill_(float("nan"))
        h = torch.cuda.current_stream().cuda_stream
        assert waits(kind, ctypes.byref(lin.struct), q.data_ptr(), ld, sx.data_ptr(), T, out.data_ptr(), err.data_ptr(),
                     limit_ns, starved, h) == _lib.MOE_OK
        torch.cuda.synchronize()
        return err.item()

    assert call(2_000_000_000, 0) == 0 and ((out.double() - ref).abs() <= tol).all()
    for _ in range(3):
        assert call(20_000_000, starve) == _lib.MOE_ERR_TIMEOUT
        assert call(2_000_000_000, 0) == 0 and ((out.double() - ref).abs() <= tol).all()
        M.moe_linear_i8(lin, q, sx, out, M.OUT_F32, err_word=err)
        torch.cuda.synchronize()
        assert err.item() == 0 and ((out.double() - ref).abs() <= tol).all()
    check_linear(4100, 1000, 450, M.OUT_F32)
    check_linear(4100, 144, 1000, M.OUT_BF16)


def test_refusals_on_the_device(cuda_ok):
    """What the quick way does not take is named by the full checks, and nothing is written."""
    lin, *_ = linear(64, 64)
    q, s, out = torch.zeros((4, 64), dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV), torch.full((4, 64), 3.0, device=DEV)
    for args, what in (((q[:, :32], s, out), "contiguous|rows hold"), ((q, s[:3], out), "qscale holds 3"),
                       ((q, s, out[:3]), "out holds"), ((q, s.double(), out), "dtype"), ((q, s, out.half()), "dtype"),
                       ((q.cpu(), s, out), "CUDA tensor"), ((q[0], s, out), r"\[T, ld\]"), ((q, s, out.T), "contiguous")):
        with pytest.raises(ValueError, match=what):
            M.moe_linear_i8(lin, *args, M.OUT_F32)
    with pytest.raises(M.MoEError):
        M.moe_linear_i8(lin, q, s, out, 5)
    with pytest.raises(M.MoEError):
        M.moe_linear_i8(lin, q.view(-1)[8:200].view(3, 64), s, out, M.OUT_F32)
    with pytest.raises(TypeError):
        M.moe_linear_i8(lin, q, [0.0], out, M.OUT_F32)
    x = torch.zeros((4, 64), device=DEV)
    for args, what in (((x.T, q, s), "contiguous"), ((x, q[:3], s), "q has 3 rows"), ((x.double(), q, s), "dtype"),
                       ((x, q, s[:2]), "scale holds 2")):
        with pytest.raises(ValueError, match=what):
            M.moe_quant_i8(*args)
    torch.cuda.synchronize()
    assert (out == 3.0).all()


def test_outputs_past_32_bit_offsets(cuda_ok):
    """More than 2^32 output elements: the last tokens and the last columns land where they belong."""
    N, K, T = 66000, 48, 65100
    lin, W, sw, b = linear(N, K, seed=9)
    g = torch.Generator(device=DEV).manual_seed(9)
    q = torch.randint(-128, 128, (T, K), dtype=torch.int8, device=DEV, generator=g)
    sx = torch.rand(T, device=DEV, generator=g) * 0.1
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    M.moe_linear_i8(lin, q, sx, out, M.OUT_BF16)
    for rows in (slice(0, 40), slice(32500, 32600), slice(T - 300, T)):
        p, ref = product64(W, sw, b, q[rows], sx[rows], K)
        tol = 3.01 * EPS32 * p.abs() + (1.01 * EPS32 + 1.01 * EPSBF) * ref.abs()
        assert ((out[rows].double() - ref).abs() <= tol).all()
    assert not torch.isnan(out[::997]).any()
