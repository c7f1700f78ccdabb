"""CPU checks of the operators around the experts: what their C entry points refuse before any launch (no GPU is touched),
their workspace sizes, and that the tests' 64-bit forms notice a planted mistake."""

import ctypes

import pytest
import torch

from quantized_mixture_experts_moe_gb300 import binding as qb
from quantized_mixture_experts_moe_gb300 import build as qbuild
from tests import block_ref as ref

ARG, UNSUPPORTED, OK = -1, -2, 0
P = 1 << 20  # an aligned address that is never read: every call here ends before a launch


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qb.lib()


def with_(base, **changes):
    d = dict(base)
    d.update(changes)
    return tuple(d.values())


PRE = dict(rows=4, cols=64, st=1, bt=1, x=P, ldx=64, w=P, eps=1e-6, n=P, ldn=64, rstd=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), ARG), (dict(cols=0), ARG), (dict(st=3), ARG), (dict(bt=-1), ARG), (dict(st=1, bt=2), ARG), (dict(st=1, bt=0), ARG),
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(n=None), ARG), (dict(ldx=63), ARG), (dict(ldn=63), ARG), (dict(x=P + 1), ARG),
    (dict(w=P + 2), ARG), (dict(rstd=P + 2), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG),
    (dict(cols=16385, ldx=16385, ldn=16385), UNSUPPORTED), (dict(rows=0, x=None, n=None), OK)])
def test_norm_pre_refuses(lib, change, want):
    assert lib.qmoe_norm_pre(*with_(PRE, **change)) == want


POST = dict(rows=4, cols=64, st=0, bt=1, r=P, ldr=64, y=P, ldy=64, w=P, mode=0, gate=None, ldg=0, alpha=1.0, w_next=P, eps=1e-6, out=P,
            ldo=64, n=P, ldn=64, rstd=P, rstd_next=P, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(mode=4), ARG), (dict(mode=-1), ARG), (dict(mode=1), ARG), (dict(mode=3, gate=P, ldg=63), ARG), (dict(mode=3, gate=P + 1, ldg=64), ARG),
    (dict(mode=1, gate=P + 2), ARG), (dict(r=None), ARG), (dict(y=None), ARG), (dict(out=None), ARG), (dict(n=None), ARG), (dict(ldr=10), ARG),
    (dict(ldn=10), ARG), (dict(out=P + 2), ARG), (dict(y=P + 1), ARG), (dict(rows=0, r=None, y=None, out=None, n=None), OK),
    (dict(cols=20000, ldr=20000, ldy=20000, ldo=20000, ldn=20000), UNSUPPORTED)])
def test_norm_post_refuses(lib, change, want):
    assert lib.qmoe_norm_post(*with_(POST, **change)) == want


def test_norm_backward_refuses(lib):
    need = lib.qmoe_norm_bwd_workspace_bytes(4, 64)
    assert need >= 3 * 4 * 64 and lib.qmoe_norm_bwd_workspace_bytes(4, 16385) == 0 == lib.qmoe_norm_bwd_workspace_bytes(-1, 8)
    pre = dict(rows=4, cols=64, st=1, bt=1, dn=P, lddn=64, x=P, ldx=64, rstd=P, w=P, dres=None, lddres=0, dx=P, lddx=64, dw=P, ws=P,
               wsn=need, stream=None)
    for change in (dict(dn=None), dict(x=None), dict(rstd=None), dict(w=None), dict(dx=None), dict(dw=None), dict(ws=None), dict(wsn=need - 1),
                   dict(ws=P + 16), dict(lddn=1), dict(dres=P, lddres=3), dict(dres=P + 1, lddres=64), dict(st=2, bt=1)):
        assert lib.qmoe_norm_pre_backward(*with_(pre, **change)) == ARG, change
    post = dict(rows=4, cols=64, st=1, bt=1, dout=P, lddout=64, y=P, ldy=64, w=P, rstd=P, mode=2, gate=P, ldg=0, alpha=1.0, dn=P, lddn=64,
                out=P, ldo=64, w_next=P, rstd_next=P, dr=P, lddr=64, dy=P, lddy=64, dw=P, dgate=P, lddg=0, dw_next=P, ws=P, wsn=need,
                stream=None)
    for change in (dict(dout=None, dn=None), dict(y=None), dict(rstd=None), dict(dw=None), dict(gate=None), dict(dgate=None), dict(out=None),
                   dict(w_next=None), dict(rstd_next=None), dict(dw_next=None), dict(dr=None), dict(dy=None), dict(mode=3, ldg=64, lddg=8),
                   dict(mode=7), dict(lddr=8), dict(wsn=0)):
        assert lib.qmoe_norm_post_backward(*with_(post, **change)) == ARG, change


ROUTE = dict(T=4, E=64, k=2, dt=1, lg=P, ld=64, bias=None, mask=None, renorm=1, scale=1.0, ids=P, w=P, lse=P, coef=0.0, counts=None, probs=None,
             loss=None, ws=None, wsn=0, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), ARG), (dict(E=0), ARG), (dict(k=0), ARG), (dict(k=65), ARG), (dict(dt=9), ARG), (dict(ld=63), ARG), (dict(scale=0.0), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG), (dict(lg=None), ARG), (dict(ids=None), ARG), (dict(w=None), ARG),
    (dict(counts=P), ARG), (dict(counts=P, probs=P, loss=P), ARG), (dict(lg=P + 1), ARG), (dict(bias=P + 1), ARG),
    (dict(counts=P, probs=P, loss=P, ws=P, wsn=8), ARG), (dict(E=1025, ld=1025), UNSUPPORTED), (dict(k=33), UNSUPPORTED),
    (dict(T=0, lg=None, ids=None, w=None), OK)])
def test_route_refuses(lib, change, want):
    assert lib.qmoe_route_topk(*with_(ROUTE, **change)) == want


def test_route_backward_refuses(lib):
    assert lib.qmoe_route_workspace_bytes(100, 64) > 0 and lib.qmoe_route_workspace_bytes(100, 1025) == 0
    base = dict(T=4, E=64, k=2, dt=1, lg=P, ld=64, ids=P, w=P, lse=P, renorm=1, scale=1.0, dw=P, coef=0.0, counts=P, dloss=P, dl=P, ldd=64,
                stream=None)
    for change in (dict(dw=None, dloss=None), dict(lg=None), dict(ids=None), dict(w=None), dict(lse=None), dict(counts=None), dict(dl=None),
                   dict(ldd=63), dict(dl=P + 1), dict(scale=-1.0)):
        assert lib.qmoe_route_topk_backward(*with_(base, **change)) == ARG, change


def mat(**changes):
    d = dict(q=P, ld=256, s=P, s_row=2, s_blk=1, s_rows=1, reserved=0)
    d.update(changes)
    return ctypes.byref(qb.Fp8Mat(*d.values()))


def test_fp8_refuses(lib):
    rows = dict(rows=4, cols=200, dt=1, x=P, ldx=200, q=P, ldq=208, s=P, stream=None)
    for change in (dict(rows=-1), dict(cols=0), dict(dt=5), dict(x=None), dict(ldx=199), dict(q=None), dict(ldq=200), dict(ldq=192),
                   dict(q=P + 8), dict(s=None), dict(s=P + 1), dict(x=P + 1)):
        assert lib.qmoe_fp8_quant_rows(*with_(rows, **change)) == ARG, change
    cols = dict(rows=4, cols=200, dt=1, x=P, ldx=200, qt=P, ldqt=16, st=P, q=None, ldq=0, s=None, stream=None)
    for change in (dict(qt=None), dict(ldqt=8), dict(st=None), dict(q=P, ldq=100), dict(q=P, ldq=208)):
        assert lib.qmoe_fp8_quant_cols(*with_(cols, **change)) == ARG, change
    blocks = dict(rows=4, cols=200, dt=1, x=P, ldx=200, q=P, ldq=208, qt=None, ldqt=0, s=P, stream=None)
    for change in (dict(q=None), dict(s=None), dict(qt=P, ldqt=3), dict(ldq=201)):
        assert lib.qmoe_fp8_quant_blocks(*with_(blocks, **change)) == ARG, change
    mm = dict(M=4, N=8, K=256, a=mat(), b=mat(), c=P, ct=1, ldc=8, st=P, stream=None)
    for change in (dict(M=-1), dict(N=0), dict(K=0), dict(ct=4), dict(ldc=7), dict(c=None), dict(c=P + 1), dict(st=None), dict(a=None), dict(b=None),
                   dict(a=mat(q=None)), dict(a=mat(ld=250)), dict(a=mat(ld=264)), dict(b=mat(q=P + 4)), dict(b=mat(s=None)), dict(b=mat(s_rows=64))):
        assert lib.qmoe_fp8_matmul(*with_(mm, **change)) == ARG, change
    assert lib.qmoe_fp8_matmul(*with_(mm, M=0)) == OK
    assert lib.qmoe_fp8_matmul(*with_(mm, M=1 << 31)) == UNSUPPORTED
    need = lib.qmoe_fp8_linear_workspace_bytes(4, 200)
    assert need >= 4 * 208 + 4 * 2 * 4 and lib.qmoe_fp8_linear_workspace_bytes(0, 8) == 0
    lin = dict(M=4, N=8, K=200, xt=1, x=P, ldx=200, w=mat(), y=P, yt=1, ldy=8, st=P, ws=P, wsn=need, stream=None)
    for change in (dict(x=None), dict(xt=7), dict(ldx=100), dict(w=None), dict(y=None), dict(ws=None), dict(wsn=need - 1), dict(ws=P + 16),
                   dict(ldy=1), dict(st=P + 1)):
        assert lib.qmoe_fp8_linear(*with_(lin, **change)) == ARG, change


def test_reference_notices_a_planted_mistake():
    # the tolerances are narrow enough to tell one wrong expert count, one code a step off, or a mean over H - 1 columns
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(4, 300, generator=g), torch.ones(300)
    n, _ = ref.norm(x.double(), w.double(), 1e-6)
    wrong = (x.double() / torch.sqrt(x.double().square().sum(-1, keepdim=True) / 299 + 1e-6)).float()
    ref.close(n.float(), n, (300 / 128 + 48) * 2.0 ** -24 * n.abs())
    with pytest.raises(AssertionError):
        ref.close(wrong, n, (300 / 128 + 48) * 2.0 ** -24 * n.abs())
    a, a_s = ref.quant(torch.randn(8, 256, generator=g), 1)
    b, b_s = ref.quant(torch.randn(8, 256, generator=g), 1)
    want, slack = ref.product(ref.dequant(a, a_s), ref.dequant(b, b_s))
    moved = a.view(torch.uint8).clone()
    moved[3, 7] ^= 1
    off, _ = ref.product(ref.dequant(moved.view(torch.float8_e4m3fn), a_s), ref.dequant(b, b_s))
    with pytest.raises(AssertionError):
        ref.close(off.float(), want, slack)
    lg = torch.randn(6, 10, generator=g).double().requires_grad_()
    one = ref.route(lg, 2, None, None, True, 1.0, 1.0)
    other = ref.route(lg, 2, None, torch.tensor([1, 1, 1, 1, 1, 0]).bool(), True, 1.0, 1.0)
    assert not torch.equal(one["counts"], other["counts"]) and abs(float((one["loss"] - other["loss"]).detach())) > 1e-4


def test_linear_backward_refuses_shapes_that_do_not_go_together():
    status = torch.zeros(1, dtype=torch.int32)
    dy, x, wt, s = torch.zeros(3, 8), torch.zeros(3, 16), torch.zeros(16, 8, dtype=torch.uint8), torch.ones(1, 1)
    for bad in [(dy[:2], x, wt, s), (dy, x[:, :8], wt, s), (dy, x, wt.t(), s), (dy[0], x, wt, s), (dy, x, wt[0], s)]:
        with pytest.raises(ValueError):
            qb.fp8_linear_backward(*bad, dev_status=status)
    with pytest.raises(qb.QmoeError, match="device"):
        qb.fp8_linear_backward(dy, x, wt, s, dev_status=status)
    with pytest.raises(qb.QmoeError, match="device"):
        qb.fp8_linear_backward(dy, x, wt, s)


def test_tensors_of_two_devices_are_refused(lib):
    # tensors that say where they lie and have no memory: a call ends before it asks for their pointers
    class Placed(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise NotImplementedError(func)

    def at(i, *shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(Placed, shape, dtype=dtype, device=torch.device("cuda", i))

    a, b = ([at(i, 4, 64), at(i, 64), at(i, 4)] for i in range(2))
    codes, scales = [at(i, 4, 64, dtype=torch.uint8) for i in range(2)], [at(i, 4, 1) for i in range(2)]
    word = [at(i, 1, dtype=torch.int32) for i in range(2)]
    r = qb.Routing()
    r.ids, r.w, r.lse, r.counts, r.renorm, r.scale, r.coef = word[0], a[1], a[2], word[0], True, 1.0, 1.0
    for call in (lambda: qb.norm_pre(a[0], b[1]),
                 lambda: qb.norm_pre_backward(a[0], a[0], a[2], a[1], dres=b[0]),
                 lambda: qb.norm_post(a[0], b[0]),
                 lambda: qb.norm_post_backward(a[0], a[0], gate=b[1]),
                 lambda: qb.route_topk(a[0], 2, bias=b[1]),
                 lambda: qb.route_topk_backward(a[0], r, dloss=b[2]),
                 lambda: qb.fp8_matmul(codes[0], scales[0], codes[1], scales[1], dev_status=word[0]),
                 lambda: qb.fp8_linear(a[0], codes[0], scales[0], dev_status=word[1]),
                 lambda: qb.fp8_linear_backward(a[0], a[0], codes[0], scales[1], dev_status=word[0])):
        with pytest.raises(qb.QmoeError, match="one device"):
            call()


def test_a_moved_package_loads_its_own_library(lib, tmp_path):
    import shutil
    import subprocess
    import sys

    shutil.copytree(qbuild.PKG, tmp_path / "quantized_mixture_experts_moe_gb300", ignore=shutil.ignore_patterns("_build", "__pycache__"))
    code = ("from quantized_mixture_experts_moe_gb300 import binding as qb\n"
            "assert qb._load_bind().__file__.startswith({0!r})\n"
            "maps = {{line.split()[-1] for line in open('/proc/self/maps') if 'libqmoe.so' in line}}\n"
            "assert len(maps) == 1 and maps.pop().startswith({0!r}), maps\n").format(str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_a_module_for_another_torch_is_built_again(lib, monkeypatch):
    assert qbuild.up_to_date()
    monkeypatch.setattr(qbuild, "bind_target", lambda: "python 3.0\ntorch 1.0\n")
    assert not qbuild.up_to_date()
