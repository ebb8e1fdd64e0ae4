"""The whole routed-expert layer for a few tokens, and the 8-bit integer matrix product: cases, plain forms and
the library's calls.

Three kinds of case:

* ``layer``: RMSNorm (where the case has it), router, top-K gating, the chosen int4 experts, the shared expert,
  LoRA and the combine, for 1 to 32 tokens: ``moe_layer_decode``.
* ``linear``: an 8-bit integer matrix product with one scale per token and one per output channel:
  ``moe_linear_i8``.
* ``proj``: a quantised projection of the residual stream as a decoder runs it, from the activations: per-token
  quantisation (after RMSNorm where the case has it), then the product: ``moe_quant_i8``, ``moe_linear_i8``.

The plain forms read the library's storage formats (``include/moe.h``): a quantised row is a record of codes, fp16
scales and fp16 biases per group of 64 inputs, an expert is one block of records.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ----------------------------------------------------------------------------- cases
def _layer(name, T, H, E, K, I, r, norm, forced=False, down_lora=False, bf16=False):
    return {"name": name, "op": "layer", "T": T, "H": H, "E": E, "K": K, "I": I, "r": r, "norm": norm,
            "forced": forced, "down_lora": down_lora, "bf16": bf16}


def _linear(name, op, T, K, N, bias, bf16, norm=False, x_bf16=False):
    return {"name": name, "op": op, "T": T, "K": K, "N": N, "bias": bias, "bf16": bf16, "norm": norm,
            "x_bf16": x_bf16}


def listed():
    return [
        # the smallest layer of the configurations: launch and exchange latency only
        _layer("layer tiny, 4 tokens", 4, 256, 16, 2, 128, 8, norm=False, bf16=True),
        # one token of one layer at the 35B shape: interactive decoding
        _layer("layer 35B, 1 token", 1, 2048, 256, 4, 512, 16, norm=True),
        # a handful of sequences at the 8B shape (eight of 128 experts each)
        _layer("layer 8B, 7 tokens", 7, 2048, 128, 8, 512, 16, norm=True),
        # a small batch without adapters at the 35B shape
        _layer("layer 35B, 16 tokens", 16, 2048, 256, 4, 512, 0, norm=False, bf16=True),
        # batched decoding on the previous layer's predicted experts, with adapters on the routed experts
        _layer("layer 35B, 32 predicted", 32, 2048, 256, 4, 512, 16, norm=True, forced=True, down_lora=True),
        # one token's projection of the residual stream (the attention projections around the layer)
        _linear("proj 1 token", "proj", 1, 2048, 4096, bias=False, bf16=True, norm=True),
        # a batched decoding step's projection
        _linear("proj 64 tokens", "proj", 64, 2048, 2048, bias=False, bf16=False, norm=True),
        # a prompt's projection
        _linear("proj 3328 tokens", "proj", 3328, 2048, 4096, bias=True, bf16=True, norm=True),
        # the output head for one token: a long weight stream
        _linear("linear head, 1 token", "linear", 1, 2048, 65536, bias=False, bf16=False),
        # odd sizes
        _linear("linear odd, 13 tokens", "linear", 13, 1000, 2051, bias=True, bf16=False),
        # the ordinary prompt product
        _linear("linear 1024 tokens", "linear", 1024, 4096, 2048, bias=False, bf16=True),
        # the largest product: compute bound
        _linear("linear 8192 tokens", "linear", 8192, 4096, 4096, bias=True, bf16=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            H, I = 2 ** rng.randint(8, 12), 2 ** rng.randint(7, 11)
            E = rng.randint(8, 256)
            K = rng.randint(1, 8)
            T = rng.randint(1, min(32, 65536 // H))
            r = rng.choice([0, 8, 16, 24, 32])
            # a pool no larger than the 35B layer's; no more work than 32 tokens of it
            if E * H * I <= 256 * 2048 * 512 and T * K * H * I <= 128 * 2048 * 512:
                break
        return {"op": "layer", "T": T, "H": H, "E": E, "K": K, "I": I, "r": r, "norm": rng.random() < 0.5,
                "forced": rng.random() < 0.3, "down_lora": r > 0 and rng.random() < 0.3, "bf16": rng.random() < 0.4}
    op = rng.choice(["linear", "proj"])
    while True:
        T, K, N = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192), _log_int(rng, 64, 65536)
        if T * K * N <= 8192 * 4096 * 4096 and K * N <= 65536 * 2048 and T * N <= 8192 * 8192:
            break
    return {"op": op, "T": T, "K": K, "N": N, "bias": rng.random() < 0.5, "bf16": rng.random() < 0.5,
            "norm": op == "proj" and rng.random() < 0.5, "x_bf16": op == "proj" and rng.random() < 0.5}


# ----------------------------------------------------------------------------- inputs
def _rec_bytes(n_in, bits):
    return (n_in * bits // 8 + 4 * (n_in // 64) + 15) // 16 * 16


def _records(g, rows, n_in, bits):
    """[*rows, record] bytes: uniform codes, scale ~ U(0.005, 0.02) (8 bits: a sixteenth of it), bias about minus
    half the code range times the scale, as a min/max grid gives them."""
    cb, G = n_in * bits // 8, n_in // 64
    rec = torch.randint(0, 256, (*rows, _rec_bytes(n_in, bits)), dtype=torch.uint8, device=DEV, generator=g)
    s = torch.rand((*rows, G), device=DEV, generator=g) * 0.015 + 0.005
    mid = 2.0 ** (bits - 1) + (torch.rand((*rows, G), device=DEV, generator=g) - 0.5) * 2.0 ** (bits - 6)
    s = (s / (1 if bits == 4 else 16)).half()
    b = (-mid * s.float()).half()
    rec[..., cb:cb + 2 * G] = s.view(torch.uint8)
    rec[..., cb + 2 * G:cb + 4 * G] = b.view(torch.uint8)
    rec[..., cb + 4 * G:] = 0
    return rec


def _blocks(g, n, H, I):
    """n expert blocks, each a multiple of 256 bytes: 2I gate/up records (interleaved), then H down records."""
    gu = _records(g, (n, 2 * I), H, 4).view(n, -1)
    dn = _records(g, (n, H), I, 4).view(n, -1)
    size = gu.shape[1] + dn.shape[1]
    out = torch.zeros((n, (size + 255) // 256 * 256), dtype=torch.uint8, device=DEV)
    out[:, :gu.shape[1]] = gu
    out[:, gu.shape[1]:size] = dn
    return out


def _adapter(g, n, H_in, H_out, r):
    A = (torch.randn((*n, r, H_in), device=DEV, generator=g) * 0.02).half()
    B = (torch.randn((*n, H_out, r), device=DEV, generator=g) * 0.02).half()
    return A, B


def _prepare_layer(c, g):
    T, H, E, K, I, r = (c[k] for k in ("T", "H", "E", "K", "I", "r"))
    s = {"case": c, "T": T, "H": H, "E": E, "K": K, "I": I, "r": r}
    s["router"] = _records(g, (E,), H, 8)
    s["router_bias"] = torch.randn(E, device=DEV, generator=g) * 0.5
    s["gate"] = _records(g, (1,), H, 8)
    s["pool"] = _blocks(g, E, H, I)
    s["shared"] = _blocks(g, 1, H, I)[0]
    s["sh_lora"] = [_adapter(g, (), H, I, r), _adapter(g, (), H, I, r), _adapter(g, (), I, H, r)] if r else None
    s["ex_lora"] = _adapter(g, (E,), I, H, r) if c["down_lora"] else None
    x = torch.randn((T, H), device=DEV, generator=g) * (0.5 + 2.0 * torch.rand((T, 1), device=DEV, generator=g))
    s["x"], s["u"] = (x, None) if c["norm"] else (None, (x / x.square().mean(1, keepdim=True).sqrt()).bfloat16())
    s["exec"] = None
    if c["forced"]:
        s["exec"] = torch.rand((T, E), device=DEV, generator=g).argsort(1)[:, :K].int().contiguous()
    if own:
        import int4_expert_ffn_top_b200 as M

        s["M"] = M
        s["layer"] = M.DeviceLayer.from_tensors(
            H=H, E=E, I=I, r=r, router=s["router"], router_bias=s["router_bias"], shared_gate=s["gate"],
            shared_block=s["shared"], pool=s["pool"], shared_lora=s["sh_lora"], routed_down_lora=s["ex_lora"])
        s["idx"] = torch.empty((T, K), dtype=torch.int32, device=DEV)
        s["w"] = torch.empty((T, K), device=DEV)
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16 if c["bf16"] else torch.float32, device=DEV)
        s["ws"] = M.workspace(M.moe_layer_decode_workspace_size(s["layer"], T, K))
    return s


def _prepare_linear(c, g):
    T, K, N = c["T"], c["K"], c["N"]
    s = {"case": c}
    s["W"] = torch.randint(-127, 128, (N, K), dtype=torch.int8, device=DEV, generator=g)
    s["w_scale"] = (0.5 + torch.rand(N, device=DEV, generator=g)) / (64 * math.sqrt(K))
    s["bias"] = torch.randn(N, device=DEV, generator=g) * 0.1 if c["bias"] else None
    if c["op"] == "proj":  # activations with a few large channels, as a residual stream has
        x = torch.randn((T, K), device=DEV, generator=g) * (1 + 9 * (torch.rand(K, device=DEV, generator=g) < 0.01))
        s["x"] = x.bfloat16() if c["x_bf16"] else x
    else:
        s["q"] = (torch.randn((T, K), device=DEV, generator=g) * 40).round().clamp(-127, 127).to(torch.int8)
        s["q_scale"] = (0.5 + torch.rand(T, device=DEV, generator=g)) / 40
    if own:
        import int4_expert_ffn_top_b200 as M

        s["M"] = M
        s["lin"] = M.DeviceLinear8(s["W"], s["w_scale"], s["bias"])
        ld = M.moe_i8_row_bytes(K)
        codes = torch.zeros((T, ld), dtype=torch.int8, device=DEV)
        if c["op"] == "proj":
            s["q_scale"] = torch.empty(T, device=DEV)
        else:
            codes[:, :K] = s["q"]
        s["codes"] = codes
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16 if c["bf16"] else torch.float32, device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (_prepare_layer if case["op"] == "layer" else _prepare_linear)(case, g)


# ----------------------------------------------------------------------------- plain forms
def _weights(rec, n_in, bits, dtype=torch.float32):
    """Dequantised matrices of records [..., rows, record]: code * scale + bias per group of 64 inputs."""
    cb, G = n_in * bits // 8, n_in // 64
    q = rec[..., :cb]
    if bits == 4:
        q = torch.stack([q & 15, q >> 4], -1).flatten(-2)
    s = rec[..., cb:cb + 2 * G].contiguous().view(torch.float16).to(dtype)
    b = rec[..., cb + 2 * G:cb + 4 * G].contiguous().view(torch.float16).to(dtype)
    q = q.to(dtype).unflatten(-1, (G, 64))
    return (q * s[..., None] + b[..., None]).flatten(-2)


def _silu(a):
    return a / (1 + torch.exp(-a))


def _ffn(u, block, H, I, lora=None):
    """SwiGLU of one block per row of u [n, H]: block [n or 1, bytes], lora gate/up/down (A, B) or None each."""
    n = block.shape[0]
    ngu = 2 * I * _rec_bytes(H, 4)
    gu = _weights(block[:, :ngu].reshape(n, 2 * I, -1), H, 4)
    dn = _weights(block[:, ngu:ngu + H * _rec_bytes(I, 4)].reshape(n, H, -1), I, 4)

    def mul(W, x):  # W [n or 1, out, in], x [rows, in]
        return torch.bmm(W, x[:, :, None])[:, :, 0] if n == x.shape[0] else x @ W[0].T

    def delta(p, x):
        if lora is None or lora[p] is None:
            return 0.0
        A, B = (t.float() for t in lora[p])
        if A.dim() == 3:
            return torch.bmm(B, torch.bmm(A, x[:, :, None]))[:, :, 0]
        return (x @ A.T) @ B.T

    ab = mul(gu, u)
    h = _silu(ab[:, 0::2] + delta(0, u)) * (ab[:, 1::2] + delta(1, u))
    return mul(dn, h) + delta(2, h)


def _plain_layer(s):
    T, H, I, K = s["T"], s["H"], s["I"], s["K"]
    if s["x"] is not None:  # in 64 bits: u's rounding and the top-K are decisions next to a border
        x = s["x"].double()
        u16 = (x / (x.square().mean(1, keepdim=True) + EPS).sqrt()).bfloat16()
    else:
        u16 = s["u"]
    u = u16.float()
    logits = u.double() @ _weights(s["router"], H, 8, torch.float64).T + s["router_bias"].double()
    idx = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :K]
    chosen = idx if s["exec"] is None else s["exec"].long()
    sel = torch.gather(logits, 1, chosen)
    w = torch.exp(sel - sel.max(1, keepdim=True)[0])
    w = (w / w.sum(1, keepdim=True)).float()
    g = 1 / (1 + torch.exp(-(u @ _weights(s["gate"], H, 8).T)))
    flat = chosen.reshape(-1)
    lora = None
    if s["ex_lora"] is not None:
        lora = (None, None, (s["ex_lora"][0][flat], s["ex_lora"][1][flat]))
    y = _ffn(u.repeat_interleave(K, 0), s["pool"][flat], H, I, lora).view(T, K, H)
    out = (w[:, :, None] * y).sum(1) + g * _ffn(u, s["shared"][None], H, I, s["sh_lora"])
    return {"out": out.bfloat16() if s["case"]["bf16"] else out, "idx": idx.int(), "w": w}


def _codes(x, norm):
    """Per-token symmetric 8-bit codes and scales; the codes are the nearest integers to 127 x / max|x|, ties to
    even, in 64 bits (a value next to a border decides a code).  RMSNorm scales a row and leaves its codes."""
    x = x.double()
    m = x.abs().amax(1, keepdim=True)
    q = torch.where(m > 0, (127 * x / m).round(), torch.zeros_like(x))
    if norm:
        m = m / (x.square().mean(1, keepdim=True) + EPS).sqrt()
    return q.float(), (m / 127).float()


def _plain_linear(s):
    if s["case"]["op"] == "proj":
        q, sx = _codes(s["x"], s["case"]["norm"])
    else:
        q, sx = s["q"].float(), s["q_scale"][:, None]
    y = (q @ s["W"].float().T) * sx * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.bfloat16() if s["case"]["bf16"] else y


# ----------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        M = s["M"]
        mode = M.OUT_BF16 if c["bf16"] else M.OUT_F32
        if c["op"] == "layer":
            M.moe_layer_decode(s["layer"], s["u"], s["K"], s["idx"], s["w"], s["out"], mode, s["ws"], x=s["x"],
                               eps=EPS, exec_idx=s["exec"])
            return {"out": s["out"], "idx": s["idx"], "w": s["w"]}
        if c["op"] == "proj":
            M.moe_quant_i8(s["x"], s["codes"], s["q_scale"], eps=EPS if c["norm"] else None)
        M.moe_linear_i8(s["lin"], s["codes"], s["q_scale"], s["out"], mode)
        return s["out"]
    return _plain_layer(s) if c["op"] == "layer" else _plain_linear(s)


# ----------------------------------------------------------------------------- floors
def work(c):
    T = c["T"]
    if c["op"] == "layer":
        H, E, K, I, r = c["H"], c["E"], c["K"], c["I"], c["r"]
        block = 2 * I * _rec_bytes(H, 4) + H * _rec_bytes(I, 4)
        D = E * (1 - (1 - K / E) ** T)  # distinct experts of T tokens, each taking K of E
        b = (D + 1) * block + (E + 1) * _rec_bytes(H, 8) + 4 * E + T * H * (4 if c["norm"] else 2)
        b += 2 * r * 3 * (H + I)  # the shared expert's three adapters, A [r, in] and B [out, r]
        b += D * 2 * r * (H + I) if c["down_lora"] else 0
        b += T * H * (2 if c["bf16"] else 4) + T * K * (12 if c["forced"] else 8)
        f = 2 * T * ((K + 1) * 3 * H * I + (E + 1) * H)
        f += 2 * T * r * (3 * H + 3 * I) + (2 * T * K * r * (H + I) if c["down_lora"] else 0)
        return {"bytes": b, "flops": f}
    K, N = c["K"], c["N"]
    b = N * K + 4 * N * (2 if c["bias"] else 1) + T * N * (2 if c["bf16"] else 4)
    b += T * K * (2 if c["x_bf16"] else 4) if c["op"] == "proj" else T * (K + 4)
    return {"bytes": b, "flops": 2 * T * N * K}


# ----------------------------------------------------------------------------- the definition in 64 bits
def _matrix64(records, n_in, bits):
    """[rows, n_in] of one matrix's records, each element from its own code, scale and bias."""
    at = torch.arange(n_in, device=records.device)
    if bits == 4:
        word = records[:, :n_in // 2].contiguous().view(torch.int32).long()
        code = (word[:, at // 8] >> (4 * (at % 8))) & 15
    else:
        code = records[:, at].long()
    halves = records[:, n_in * bits // 8:].contiguous().view(torch.float16).double()
    return code * halves[:, at // 64] + halves[:, n_in // 64 + at // 64]


def _expert64(u, block, H, I, gate=None, up=None, down=None):
    cut = 2 * I * _rec_bytes(H, 4)
    W = _matrix64(block[:cut].view(2 * I, -1), H, 4)
    D = _matrix64(block[cut:cut + H * _rec_bytes(I, 4)].view(H, -1), I, 4)
    for adapter, rows in ((gate, W[0::2]), (up, W[1::2]), (down, D)):
        if adapter is not None:
            rows += adapter[1].double() @ adapter[0].double()
    a, b = u @ W[0::2].T, u @ W[1::2].T
    return (a * torch.sigmoid(a) * b) @ D.T


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "layer":
        N = s["W"].shape[0]
        if case["op"] == "proj":
            x = s["x"].double()
            top = x.abs().max(1)[0]
            unit = torch.where(top > 0, top / 127, torch.ones_like(top))
            q = torch.round(x * 127 / (unit * 127)[:, None])
            if case["norm"]:
                unit = unit * torch.rsqrt((x * x).sum(1) / x.shape[1] + EPS)
        else:
            q, unit = s["q"].double(), s["q_scale"].double()
        y = torch.empty((q.shape[0], N), dtype=torch.float64, device=DEV)
        for n in range(0, N, 8192):
            y[:, n:n + 8192] = unit[:, None] * (q @ s["W"][n:n + 8192].double().T * s["w_scale"][n:n + 8192].double())
        return y if s["bias"] is None else y + s["bias"].double()
    T, H, I, K = s["T"], s["H"], s["I"], s["K"]
    if s["x"] is not None:
        x = s["x"].double()
        u = (x * torch.rsqrt((x * x).sum(1, keepdim=True) / H + EPS)).to(torch.bfloat16).double()
    else:
        u = s["u"].double()
    logits = u @ _matrix64(s["router"], H, 8).T + s["router_bias"]
    idx = torch.argsort(-logits, dim=1, stable=True)[:, :K]
    chosen = idx if s["exec"] is None else s["exec"].long()
    w = torch.softmax(torch.gather(logits, 1, chosen), 1)
    sh = s["sh_lora"] or (None, None, None)
    out = torch.sigmoid(u @ _matrix64(s["gate"], H, 8).T) * _expert64(u, s["shared"], H, I, *sh)
    for e in torch.unique(chosen).tolist():
        t, k = torch.nonzero(chosen == e, as_tuple=True)
        down = None if s["ex_lora"] is None else (s["ex_lora"][0][e], s["ex_lora"][1][e])
        out.index_put_((t,), w[t, k][:, None] * _expert64(u[t], s["pool"][e], H, I, down=down), accumulate=True)
    return {"out": out, "idx": None, "w": w}
