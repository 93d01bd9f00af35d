"""Sequence operators without a GPU: refusals of the C ABI before any launch,
workspace queries, and the fp64 reference against autograd and differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

from depthwise_convolution_grouped_amd import gconv as G
from depthwise_convolution_grouped_amd import seq
from oracle import seq as ref

P = 4096   # an address that no refused call may touch


def glr_desc(B=2, L=10, D=6, dtype=G.GCONV_BF16, c=8.0, **strides):
    d = G.gconv_glr_desc(dtype=dtype, c=c, B=B, L=L, D=D)
    for name in ("x", "r", "i", "y", "dx", "dr", "di"):
        setattr(d, name + "_stride", (ctypes.c_int64 * 2)(*strides.get(name, (L * D, D))))
    return d


def fwd(d, x=P, r=P, i=P, lam=P, h0=None, lengths=None, y=P, h_last=None, states=None):
    return G.lib().gconv_glr_fwd(ctypes.byref(d) if d else None, x, r, i, lam, h0, lengths, y, h_last, states,
                                 None, 0, None)


def bwd(d, x=P, r=P, i=P, lam=P, lengths=None, states=P, dy=P, dh=None, dx=P, dr=P, di=P, dlam=P, dh0=None, ws=P,
        nbytes=0):
    return G.lib().gconv_glr_bwd(ctypes.byref(d) if d else None, x, r, i, lam, lengths, states, dy, dh, dx, dr, di,
                                 dlam, dh0, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), G.GCONV_ERR_BAD_DESC),
    (dict(c=0.0), G.GCONV_ERR_BAD_DESC),
    (dict(c=-1.0), G.GCONV_ERR_BAD_DESC),
    (dict(c=math.inf), G.GCONV_ERR_BAD_DESC),
    (dict(c=math.nan), G.GCONV_ERR_BAD_DESC),
    (dict(B=-1), G.GCONV_ERR_BAD_DESC),
    (dict(L=-1), G.GCONV_ERR_BAD_DESC),
    (dict(D=0), G.GCONV_ERR_BAD_DESC),
    (dict(B=1 << 31, L=1, y=(6, 6)), G.GCONV_ERR_TOO_LARGE),
    (dict(B=1, L=1 << 31), G.GCONV_ERR_TOO_LARGE),
    (dict(B=1, L=1, D=1 << 31), G.GCONV_ERR_TOO_LARGE),
    (dict(x=(-60, 6)), G.GCONV_ERR_BAD_DESC),
    (dict(r=(60, -6)), G.GCONV_ERR_BAD_DESC),
    (dict(i=(60, 1 << 41)), G.GCONV_ERR_BAD_DESC),
    (dict(y=(60, 5)), G.GCONV_ERR_BAD_DESC),     # rows overlap
    (dict(y=(0, 6)), G.GCONV_ERR_BAD_DESC),      # batch rows overlap
    (dict(y=(59, 6)), G.GCONV_ERR_BAD_DESC),
    (dict(y=(6, 11)), G.GCONV_ERR_BAD_DESC),     # time-major, two batch rows of 6 in 11
])
def test_recurrence_refuses_bad_descriptors(kw, status):
    d = glr_desc(**kw)
    assert fwd(d) == status
    n = ctypes.c_size_t()
    assert G.lib().gconv_glr_fwd_workspace(ctypes.byref(d), ctypes.byref(n)) == status


@pytest.mark.parametrize("extent,status", [((1 << 31) - 1024, G.GCONV_OK), ((1 << 31) - 1023, G.GCONV_ERR_TOO_LARGE),
                                           ((1 << 31) - 1, G.GCONV_ERR_TOO_LARGE)])
def test_extents_leave_room_for_a_block(extent, status):
    """The kernels' indices run past an extent by up to a block and must stay in an int."""
    n = ctypes.c_size_t()
    d = glr_desc(B=1, L=extent, D=1, x=(0, 0), r=(0, 0), i=(0, 0), y=(0, 1))
    assert G.lib().gconv_glr_fwd_workspace(ctypes.byref(d), ctypes.byref(n)) == status
    d = mm_desc(M=33, N=extent, K=16, w=0)
    assert G.lib().gconv_matmul_q8_workspace(ctypes.byref(d), ctypes.byref(n)) == status
    assert norm(q8_desc(M=1, D=extent, q=extent, total=extent), x=None) == (
        G.GCONV_ERR_NULL_PTR if status == G.GCONV_OK else status)


@pytest.mark.parametrize("L,D,forward,backward", [
    (9, (1 << 29) - 64, G.GCONV_OK, G.GCONV_OK), (9, (1 << 29) - 63, G.GCONV_ERR_TOO_LARGE, G.GCONV_ERR_TOO_LARGE),
    (9, (1 << 30) + 64, G.GCONV_ERR_TOO_LARGE, G.GCONV_ERR_TOO_LARGE),
    (8, (1 << 31) - 1024, G.GCONV_OK, G.GCONV_ERR_TOO_LARGE)])
def test_channels_of_a_row_fit_a_launch(L, D, forward, backward):
    """A launch holds fewer than 2^32 work-items, 8 for each channel but in the kernel of up to eight steps; the
    channels' byte offsets, which are 32-bit there, do not wrap below that."""
    n = ctypes.c_size_t()
    d = glr_desc(B=1, L=L, D=D, dtype=G.GCONV_F32, **{k: (0, D) for k in ("x", "r", "i", "y", "dx", "dr", "di")})
    assert G.lib().gconv_glr_fwd_workspace(ctypes.byref(d), ctypes.byref(n)) == forward
    assert G.lib().gconv_glr_bwd_workspace(ctypes.byref(d), ctypes.byref(n), None) == backward


def test_recurrence_takes_time_major_and_repeated_rows():
    n = ctypes.c_size_t()
    for kw in (dict(y=(6, 12)), dict(x=(0, 6)), dict(x=(60, 0)), dict(B=0), dict(L=0), dict(y=(100, 7))):
        assert G.lib().gconv_glr_fwd_workspace(ctypes.byref(glr_desc(**kw)), ctypes.byref(n)) == G.GCONV_OK, kw


def test_recurrence_refuses_bad_pointers():
    d = glr_desc()
    assert fwd(None) == G.GCONV_ERR_NULL_PTR
    for k in ("x", "r", "i", "lam", "y"):
        assert fwd(d, **{k: None}) == G.GCONV_ERR_NULL_PTR, k
        assert fwd(d, **{k: P + 1}) == G.GCONV_ERR_MISALIGNED, k
    for k in ("h0", "lengths", "h_last", "states"):
        assert fwd(d, **{k: P + 2}) == G.GCONV_ERR_MISALIGNED, k
    assert fwd(glr_desc(B=0), x=None, r=None, i=None, lam=None, y=None) == G.GCONV_OK   # nothing to do


def test_recurrence_backward_refusals():
    d = glr_desc()
    n, least = ctypes.c_size_t(), ctypes.c_size_t()
    assert G.lib().gconv_glr_bwd_workspace(ctypes.byref(d), ctypes.byref(n), ctypes.byref(least)) == G.GCONV_OK
    assert n.value >= least.value == 2 * 6 * 4
    assert bwd(d, nbytes=least.value - 1) == G.GCONV_ERR_WORKSPACE
    assert bwd(d, ws=None, nbytes=1 << 20) == G.GCONV_ERR_WORKSPACE
    assert bwd(None) == G.GCONV_ERR_NULL_PTR
    for k in ("x", "r", "i", "lam", "states", "dy", "dx", "dr", "di", "dlam"):
        assert bwd(d, nbytes=1 << 20, **{k: None}) == G.GCONV_ERR_NULL_PTR, k
        assert bwd(d, nbytes=1 << 20, **{k: P + 1}) == G.GCONV_ERR_MISALIGNED, k
    for k in ("dx", "dr", "di"):
        assert bwd(glr_desc(**{k: (0, 6)}), nbytes=1 << 20) == G.GCONV_ERR_BAD_DESC, k
    assert bwd(glr_desc(dtype=-1), nbytes=1 << 20) == G.GCONV_ERR_BAD_DESC


def test_recurrence_workspace_splits_only_few_rows():
    n = ctypes.c_size_t()

    def size(**kw):
        assert G.lib().gconv_glr_fwd_workspace(ctypes.byref(glr_desc(**kw)), ctypes.byref(n)) == G.GCONV_OK
        return n.value

    def packed(B, L, D):
        return dict(B=B, L=L, D=D, x=(L * D, D), r=(L * D, D), i=(L * D, D), y=(L * D, D))

    assert size(**packed(1, 1, 2048)) == 0
    assert size(**packed(1, 16384, 256)) > 0
    assert size(**packed(64, 4096, 4096)) == 0


def q8_desc(M=3, D=8, dtype=G.GCONV_F16, eps=1e-6, x=8, res=8, total=8, q=8):
    return G.gconv_q8_desc(dtype=dtype, eps=eps, M=M, D=D, x_stride=x, residual_stride=res, sum_stride=total,
                           q_stride=q)


def norm(d, x=P, res=P, w=P, q=P, scale=P, total=P):
    return G.lib().gconv_rmsnorm_q8(ctypes.byref(d) if d else None, x, res, w, q, scale, total, None)


def quant(d, x=P, q=P, scale=P):
    return G.lib().gconv_quant_q8(ctypes.byref(d) if d else None, x, q, scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=9), G.GCONV_ERR_BAD_DESC), (dict(M=-1), G.GCONV_ERR_BAD_DESC), (dict(D=0), G.GCONV_ERR_BAD_DESC),
    (dict(eps=-1.0), G.GCONV_ERR_BAD_DESC), (dict(eps=math.nan), G.GCONV_ERR_BAD_DESC),
    (dict(eps=math.inf), G.GCONV_ERR_BAD_DESC),
    (dict(x=-8), G.GCONV_ERR_BAD_DESC), (dict(res=-8), G.GCONV_ERR_BAD_DESC), (dict(q=7), G.GCONV_ERR_BAD_DESC),
    (dict(total=7), G.GCONV_ERR_BAD_DESC), (dict(M=1 << 31), G.GCONV_ERR_TOO_LARGE),
    (dict(D=1 << 31, q=1 << 31, total=1 << 31), G.GCONV_ERR_TOO_LARGE),
])
def test_norm_refuses_bad_descriptors(kw, status):
    assert norm(q8_desc(**kw)) == status


def test_norm_and_quant_refuse_bad_pointers():
    d = q8_desc()
    assert norm(None) == quant(None) == G.GCONV_ERR_NULL_PTR
    for k in ("x", "w", "q", "scale"):
        assert norm(d, **{k: None}) == G.GCONV_ERR_NULL_PTR, k
    assert norm(d, res=None) == G.GCONV_ERR_BAD_DESC     # a sum of one thing
    for k in ("x", "res", "w", "scale", "total"):
        assert norm(d, **{k: P + 1}) == G.GCONV_ERR_MISALIGNED, k
    for k in ("x", "q", "scale"):
        assert quant(d, **{k: None}) == G.GCONV_ERR_NULL_PTR, k
    assert norm(q8_desc(M=0), x=None, w=None, q=None, scale=None) == G.GCONV_OK
    assert quant(q8_desc(M=0), x=None, q=None, scale=None) == G.GCONV_OK


def mm_desc(M=3, N=5, K=7, dtype=G.GCONV_F16, a=None, w=None, y=None, reserved=0):
    return G.gconv_mm_q8_desc(dtype=dtype, reserved=reserved, M=M, N=N, K=K, a_stride=K if a is None else a,
                              w_stride=K if w is None else w, y_stride=N if y is None else y)


def product(d, a=P, sa=P, w=P, sw=P, bias=None, y=P):
    return G.lib().gconv_matmul_q8(ctypes.byref(d) if d else None, a, sa, w, sw, bias, y, None, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), G.GCONV_ERR_BAD_DESC), (dict(reserved=1), G.GCONV_ERR_BAD_DESC),
    (dict(M=-1), G.GCONV_ERR_BAD_DESC), (dict(N=0), G.GCONV_ERR_BAD_DESC), (dict(K=0), G.GCONV_ERR_BAD_DESC),
    (dict(K=131072), G.GCONV_ERR_TOO_LARGE),            # 131072 * 128 * 128 = 2^31
    (dict(M=1 << 31), G.GCONV_ERR_TOO_LARGE), (dict(N=1 << 31), G.GCONV_ERR_TOO_LARGE),
    (dict(a=-7), G.GCONV_ERR_BAD_DESC), (dict(w=-7), G.GCONV_ERR_BAD_DESC), (dict(y=4), G.GCONV_ERR_BAD_DESC),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1), G.GCONV_ERR_TOO_LARGE),
])
def test_product_refuses_bad_descriptors(kw, status):
    d = mm_desc(**kw)
    assert product(d) == status
    n = ctypes.c_size_t()
    assert G.lib().gconv_matmul_q8_workspace(ctypes.byref(d), ctypes.byref(n)) == status


def test_product_refuses_bad_pointers():
    d = mm_desc()
    assert product(None) == G.GCONV_ERR_NULL_PTR
    for k in ("a", "sa", "w", "sw", "y"):
        assert product(d, **{k: None}) == G.GCONV_ERR_NULL_PTR, k
    for k in ("sa", "sw", "bias", "y"):
        assert product(d, **{k: P + 1}) == G.GCONV_ERR_MISALIGNED, k
    assert product(mm_desc(M=0), a=None, sa=None, w=None, sw=None, y=None) == G.GCONV_OK


def kernel(d, a=P, w=P, workspace=True):
    n = ctypes.c_size_t()
    assert G.lib().gconv_matmul_q8_workspace(ctypes.byref(d), ctypes.byref(n)) == G.GCONV_OK
    return G.lib().gconv_matmul_q8_kernel(ctypes.byref(d), a, w, P if workspace else None, n.value).decode()


@pytest.mark.parametrize("K", list(range(1, 16)))
def test_rows_shorter_than_a_load_stay_with_the_kernel_that_takes_them(K):
    """few_any_k reads the 16 bytes that end with a row's; a shorter row has none before it."""
    for M in (1, 15, 16, 33, 64, 300, 2048, 100000):
        for N in (1, 17, 1000, 4096):
            for stride in (K, K + 1, 64):
                for at in (P, P + 1):
                    for ws in (False, True):
                        name = kernel(mm_desc(M=M, N=N, K=K, a=stride, w=stride), a=at, w=at, workspace=ws)
                        assert name == "any_k" or name.startswith("pack_k, ") and ws, (M, N, stride, name)


def test_kernel_names():
    assert kernel(mm_desc(M=1, N=64, K=32)) == "few_k 8"
    assert kernel(mm_desc(M=1, N=64, K=32), a=P + 1) == "few_any_k 16"
    for d in (mm_desc(M=0), mm_desc(K=0), mm_desc(M=1 << 31)):
        assert G.lib().gconv_matmul_q8_kernel(ctypes.byref(d), P, P, None, 0) == b""
    assert G.lib().gconv_matmul_q8_kernel(None, P, P, None, 0) == b""


def test_status_of_the_workspace():
    assert G.gconv_status_str(G.GCONV_ERR_WORKSPACE) != G.gconv_status_str(-99)


def test_wrappers_refuse_tensors_off_the_gpu():
    t = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="GPU"):
        seq.glr_fwd(t, t, t, torch.zeros(4))
    with pytest.raises(ValueError, match="GPU"):
        seq.rmsnorm_q8(t[0], torch.ones(4))
    with pytest.raises(ValueError, match="GPU"):
        seq.matmul_q8(t[0].to(torch.int8), torch.ones(3), t[0].to(torch.int8), torch.ones(3))


# ------------------------------------------------ the reference's own proofs


def _loop(x, r, i, lam, h0, lengths, c):
    """The recurrence in torch, step by step, for autograd."""
    ys, last = [], []
    for b in range(x.shape[0]):
        h, row = h0[b], []
        for t in range(x.shape[1]):
            if t < lengths[b]:
                la = -c * torch.nn.functional.softplus(lam) * torch.sigmoid(r[b, t])
                h = torch.exp(la) * h + torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(i[b, t]) * x[b, t]
                row.append(h)
            else:
                row.append(torch.zeros_like(h))
        ys.append(torch.stack(row))
        last.append(h)
    return torch.stack(ys), torch.stack(last)


def test_reference_gradient_is_autograds_and_that_of_differences():
    g = torch.Generator().manual_seed(3)
    B, L, D, c = 3, 9, 4, 5.0
    t = [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_() for s in
         ((B, L, D), (B, L, D), (B, L, D), (D,), (B, D))]
    lengths = [9, 0, 5]
    dy, dh = torch.randn(B, L, D, generator=g, dtype=torch.float64), torch.randn(B, D, generator=g, dtype=torch.float64)
    y, last = _loop(*t, lengths, c)
    (y * dy).sum().add((last * dh).sum()).backward()
    v = [k.detach().numpy() for k in t]
    f = ref.glr_fwd(*v[:4], v[4], lengths, c)
    np.testing.assert_allclose(f["y"], y.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(f["h_last"], last.detach().numpy(), rtol=1e-12, atol=1e-13)
    o = ref.glr_bwd(dy.numpy(), *v[:4], v[4], lengths, dh.numpy(), c)
    for name, k in zip(("dx", "dr", "di", "dlam", "dh0"), t):
        np.testing.assert_allclose(o[name], k.grad.numpy(), rtol=1e-10, atol=1e-12, err_msg=name)

    def loss(args):
        q = ref.glr_fwd(*args[:4], args[4], lengths, c)
        return (q["y"] * dy.numpy()).sum() + (q["h_last"] * dh.numpy()).sum()

    rng = np.random.default_rng(1)
    for k, name in enumerate(("dx", "dr", "di", "dlam", "dh0")):
        w = rng.standard_normal(v[k].shape)
        step = 1e-5
        up, down = list(v), list(v)
        up[k], down[k] = v[k] + step * w, v[k] - step * w
        # central differences: step^2 of truncation, 1e-16 / step of rounding
        assert abs((loss(up) - loss(down)) / (2 * step) - (o[name] * w).sum()) < 1e-7, name
