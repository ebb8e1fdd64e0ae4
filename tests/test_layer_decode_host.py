"""CPU checks of the whole-layer call: refusals before any launch, workspace sizes, the binding's argument order, and
DeviceLayer.from_tensors."""
import ctypes

import pytest
import torch

import int4_expert_ffn_top_b200 as M
from int4_expert_ffn_top_b200 import _lib
from int4_expert_ffn_top_b200 import build as B
from test_binding_checks import E, FakeLayer, H, K, T, cu, f32, i32, rec, u16, ws  # noqa: F401  (fixture)

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    B.build()
    return _lib.load()


def layer(**kw):
    L = _lib.moe_layer()
    L.H, L.E, L.I, L.I_s, L.r = 2048, 256, 512, 512, 16
    L.router = _lib.moe_qrows(A, 256, 2048, 8)
    L.shared_gate = _lib.moe_qrows(A, 1, 2048, 8)
    L.shared_block, L.pool, L.expert_stride = A, A, 1769472
    for k, v in kw.items():
        setattr(L, k, v)
    return L


def call(lib, L=None, u=A, x=None, eps=1e-6, T=1, K=4, idx=A, w=A, out=A, mode=0, work=A, n=1 << 30):
    L = layer() if L is None else L
    return lib.moe_layer_decode(ctypes.byref(L), u, x, eps, T, K, None, None, idx, w, out, mode, work, n, None, None)


def test_refusals(lib):
    bad, uns, small = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
    assert lib.moe_layer_decode(None, A, None, 0.0, 1, 4, None, None, A, A, A, 0, A, 1 << 20, None, None) == bad
    assert call(lib, T=0, u=None, idx=None, w=None, out=None, work=None, n=0) == _lib.MOE_OK
    for kw in (dict(u=None), dict(u=A + 8), dict(x=A + 4), dict(x=A, eps=-1.0), dict(x=A, eps=float("nan")),
               dict(idx=None), dict(w=None), dict(out=None), dict(mode=3), dict(mode=-1), dict(work=None),
               dict(work=A + 128)):
        assert call(lib, **kw) == bad, kw
    for kw in (dict(T=-1), dict(T=33), dict(K=0), dict(K=9)):
        assert call(lib, **kw) == uns, kw
    assert call(lib, n=lib.moe_layer_decode_workspace_size(ctypes.byref(layer()), 1, 4) - 1) == small
    for kw in (dict(pool=None), dict(pool=A + 16), dict(expert_stride=1769472 - 256), dict(shared_block=None),
               dict(ex_lora_A=A), dict(ex_lora_A_gu=A, ex_lora_B_gu=A + 2)):
        assert call(lib, layer(**kw)) == bad, kw
    for kw in (dict(H=2000), dict(I=500), dict(r=12), dict(E=3)):
        assert call(lib, layer(**kw)) == uns, kw


def test_addresses_that_no_element_can_have(lib):
    """fp32 and int32 at multiples of 4 bytes, bf16 of 2: the kernels' accesses would fault on anything else."""
    L = layer()
    ok = dict(ex=None, logits=None, idx=A, w=A, out=A, mode=0, err=None)

    def call(L=L, **kw):
        a = ok | kw
        return lib.moe_layer_decode(ctypes.byref(L), A, None, 0.0, 2, 4, a["ex"], a["logits"], a["idx"], a["w"], a["out"],
                                    a["mode"], A, 16, a["err"], None)

    far = A + 4096
    for kw in (dict(ex=far + 2), dict(logits=far + 1), dict(idx=A + 2), dict(w=A + 1), dict(out=A + 2), dict(out=A + 2, mode=2),
               dict(out=A + 1, mode=1), dict(err=far + 2), dict(L=layer(router_bias=A + 2))):
        assert call(**kw) == _lib.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(ex=far + 4), dict(logits=far + 4), dict(out=A + 4), dict(out=A + 2, mode=1), dict(err=far + 4)):
        assert call(**kw) == _lib.MOE_ERR_WORKSPACE, kw  # as far as the workspace check


def test_given_experts_apart_from_the_routers(lib):
    """exec_idx is read by every CTA after idx is written by one: the two may not overlap."""
    L = layer()
    for at in (A, A + 4, A + 28, A - 28):
        assert lib.moe_layer_decode(ctypes.byref(L), A, None, 0.0, 2, 4, at, None, A, A, A, 0, A, 1 << 30, None,
                                    None) == _lib.MOE_ERR_INVALID_ARG
    for at in (A + 32, A - 32):  # as far as the workspace check
        assert lib.moe_layer_decode(ctypes.byref(L), A, None, 0.0, 2, 4, at, None, A, A, A, 0, A, 16, None,
                                    None) == _lib.MOE_ERR_WORKSPACE


def test_workspace_size(lib):
    size = lambda t, k=4, **kw: lib.moe_layer_decode_workspace_size(ctypes.byref(layer(**kw)), t, k)  # noqa: E731
    assert lib.moe_layer_decode_workspace_size(None, 1, 4) == 0 and size(-1) == size(33) == size(1, 0) == 0
    assert 0 < size(1) < size(32) and size(32) % 256 == 0
    # hidden values of every slot and token, hi and lo
    assert size(32) >= (32 * 4 + 32) * 2 * 512 * 2
    assert size(4, ex_lora_A=A, ex_lora_B=A) > size(4)


@pytest.mark.parametrize("T", [1, 4, 9, 32])
@pytest.mark.parametrize("kw", [dict(ex_lora_A=A, ex_lora_B=A), dict(ex_lora_A_gu=A, ex_lora_B_gu=A)])
def test_stack_workspace_holds_every_layers(lib, T, kw):
    """A stack whose later layers alone have routed adapters needs as much as one where all of them do."""
    def size(*layers):
        return lib.moe_stack_workspace_size((_lib.moe_layer * len(layers))(*layers), None, len(layers), T, 4, 4)

    assert size(layer(), layer(**kw), layer()) == size(layer(**kw), layer(**kw), layer(**kw))
    assert size(layer(), layer(**kw)) >= lib.moe_layer_decode_workspace_size(ctypes.byref(layer(**kw)), T, 4)


def test_stack_refuses_before_its_first_layer(lib):
    """What moe_layer_decode refuses of a stack's buffers, path 4 refuses before anything is enqueued (here there is no
    device to enqueue on: MOE_ERR_CUDA)."""
    layers = (_lib.moe_layer * 3)(*[layer() for _ in range(3)])
    head = _lib.moe_prerouter(A, A, A, A, 2048, 256, 64, 256)
    heads = (_lib.moe_prerouter * 3)(head, head, head)
    T, K, row = 2, 4, 2 * 4 * 4

    def call(x=A, u=None, eps=1e-6, true=None, pred=None, path=4):
        o = _lib.moe_stack_opts(0, path, 0, 0, None)
        return lib.moe_stack_decode(layers, heads, 3, T, K, K, eps, x, None, u, None, true, pred, 1, A, ctypes.byref(o),
                                    A, 1 << 30, None)

    for kw in (dict(x=A + 4), dict(x=A + 8), dict(u=A + 8), dict(eps=-1.0), dict(eps=float("nan")),
               dict(true=A, pred=A + row), dict(true=A, pred=A + row + 4), dict(true=A, pred=A + 4)):
        assert call(**kw) == _lib.MOE_ERR_INVALID_ARG, kw
    if not torch.cuda.is_available():
        for kw in (dict(), dict(u=A), dict(true=A, pred=A), dict(true=A, pred=A + 2 * row), dict(true=A + 3 * row, pred=A)):
            assert call(**kw) == _lib.MOE_ERR_CUDA, kw


def test_binding_order_and_checks(rec):  # noqa: F811
    u, idx, w, out, work = u16(), i32(T, K), f32(T, K), f32(T, H), ws()
    M.moe_layer_decode(FakeLayer(), u, K, idx, w, out, M.OUT_F32, work, stream=0)
    name, a = rec.calls[-1]
    assert name == "moe_layer_decode"
    assert a[1:] == (u.data_ptr(), None, 1e-6, T, K, None, None, idx.data_ptr(), w.data_ptr(), out.data_ptr(), 0,
                     work.data_ptr(), 4096, None, 0)
    x, ex, lg, err = f32(T, H), i32(T, K), f32(T, E), i32(1)
    M.moe_layer_decode(FakeLayer(), None, K, idx, w, u, M.OUT_BF16, work, x=x, eps=1e-5, exec_idx=ex, logits=lg,
                       err_word=err, stream=0)
    assert rec.calls[-1][1][1:] == (None, x.data_ptr(), 1e-5, T, K, ex.data_ptr(), lg.data_ptr(), idx.data_ptr(),
                                    w.data_ptr(), u.data_ptr(), 1, work.data_ptr(), 4096, err.data_ptr(), 0)
    n = len(rec.calls)
    for kw in (dict(u=None), dict(u=u16(width=H + 64)), dict(u=f32(T, H)), dict(idx=i32(T - 1, K)), dict(w=i32(T, K)),
               dict(out=f32(T, H - 1)), dict(x=f32(T, H + 1)), dict(x=f32(T, H), u=u16(rows=T - 1)),
               dict(exec_idx=f32(T, K)), dict(logits=f32(T, E - 1)), dict(work=torch.zeros(4096, dtype=torch.uint8))):
        a = dict(u=u, idx=idx, w=w, out=out, work=work, x=None, exec_idx=None, logits=None) | kw
        with pytest.raises((ValueError, TypeError)):
            M.moe_layer_decode(FakeLayer(), a["u"], K, a["idx"], a["w"], a["out"], 0, a["work"], x=a["x"],
                               exec_idx=a["exec_idx"], logits=a["logits"], stream=0)
    assert len(rec.calls) == n


def test_layer_of_another_device_is_refused(rec):  # noqa: F811
    class There(FakeLayer):
        device = torch.device("cuda", 1)

    u, idx, w, out, work = u16(), i32(T, K), f32(T, K), f32(T, H), ws()
    for stream in (None, 0):
        with pytest.raises(ValueError, match="layer is on cuda:1"):
            M.moe_layer_decode(There(), u, K, idx, w, out, M.OUT_F32, work, stream=stream)
    slots = object.__new__(M.TieredPool)
    slots.struct = FakeLayer().struct
    with pytest.raises(ValueError, match="TieredPool"):
        M.moe_layer_decode(slots, u, K, idx, w, out, M.OUT_F32, work, stream=0)
    assert not rec.calls


def test_layer_from_tensors():
    h, e, i, r = 256, 4, 128, 8
    t = dict(router=torch.zeros((e, M.qrow_bytes(h, 8)), dtype=torch.uint8),
             shared_gate=torch.zeros((1, M.qrow_bytes(h, 8)), dtype=torch.uint8),
             shared_block=torch.zeros(M.block_stride(h, i), dtype=torch.uint8),
             pool=torch.zeros((e, M.block_stride(h, i) + 256), dtype=torch.uint8))
    if t["pool"].data_ptr() % 256:  # host allocations are 64-byte aligned
        flat = torch.zeros(t["pool"].numel() + 256, dtype=torch.uint8)
        off = -flat.data_ptr() % 256
        t["pool"] = flat[off:off + t["pool"].numel()].view(t["pool"].shape)

    def ab(*shape):
        return torch.zeros(shape, dtype=torch.float16)

    sh = [(ab(r, h), ab(i, r)), None, (ab(r, i), ab(h, r))]
    L = M.DeviceLayer.from_tensors(H=h, E=e, I=i, r=r, shared_lora=sh, routed_down_lora=(ab(e, r, i), ab(e, h, r)),
                                   lora_scale=0.5, **t)
    s = L.struct
    assert (s.H, s.E, s.I, s.I_s, s.r, s.expert_stride, s.lora_scale) == (h, e, i, i, r, t["pool"].shape[1], 0.5)
    assert s.pool == t["pool"].data_ptr() and s.sh_lora_A[0] == sh[0][0].data_ptr() and s.sh_lora_A[1] is None
    assert s.router_bias is None and s.ex_lora_A and not s.ex_lora_A_gu
    assert L.device == t["pool"].device
    for bad in (dict(router=t["router"][:-1]), dict(pool=t["pool"][:, :-16]), dict(shared_block=t["shared_block"][:512]),
                dict(shared_lora=[(ab(r, h), ab(i, r + 1)), None, None]), dict(router_bias=torch.zeros(e + 1)),
                dict(routed_down_lora=(ab(e, r, i).float(), ab(e, h, r)))):
        with pytest.raises(ValueError):
            M.DeviceLayer.from_tensors(**(dict(H=h, E=e, I=i, r=r, **t) | bad))
