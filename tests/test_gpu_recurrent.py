"""The recurrent layer: prompts against fp64 from its own 8-bit codes, tokens
against prompts, and the training step's middle against the oracles."""
import numpy as np
import pytest
import torch

import oracle
from depthwise_convolution_grouped_amd import gconv as G
from depthwise_convolution_grouped_amd import recurrent, seq
from oracle import seq as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    G.lib()


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def layer(E=48, D=40):
    return recurrent.RecurrentLayer(E, D, dtype=torch.float32, seed=3)


def conv64(u, l):
    """The causal convolution in fp64 and the sum of its terms' magnitudes."""
    B, L, D = u.shape
    w, b = f64(l.conv_w), f64(l.conv_b)
    p = np.concatenate([np.zeros((B, l.taps - 1, D)), u], 1)
    y = sum(p[:, k:k + L] * w[:, k] for k in range(l.taps)) + b
    return y, sum(np.abs(p[:, k:k + L] * w[:, k]) for k in range(l.taps)) + np.abs(b)


def test_prompt_from_its_own_codes():
    """fp64 from the norm's codes on.  The convolution's fp32 share is 1e-5 of its terms' magnitudes; the state is
    linear in its input with coefficients >= 0, so that share reaches it through the same recurrence.  A code of the
    outgoing rows may be off by one where its value lies within 1e-3 of a border."""
    l = layer()
    B, L, E = 3, 150, 48
    g = torch.Generator(device="cuda").manual_seed(5)
    x, res = (torch.randn(B, L, E, device="cuda", generator=g) for _ in range(2))
    n = torch.tensor([150, 2, 77], dtype=torch.int32, device="cuda")
    out, total, state = l.prompt(x, res, lengths=n)
    q, s, t2 = seq.rmsnorm_q8(x.view(B * L, E), l.norm, residual=res.view(B * L, E))
    assert torch.equal(total.view(B * L, E), t2)
    rows = [ref.matmul_q8(q.cpu().numpy(), f64(s), w[0].cpu().numpy(), f64(w[1]))[0] for w in (l.w_u, l.w_g)]
    u, gates = rows[0].reshape(B, L, l.D), rows[1].reshape(B, L, 3 * l.D)
    r, i, gate = (gates[..., k * l.D:(k + 1) * l.D] for k in range(3))
    c, mag = conv64(u, l)
    lam = f64(l.lam)
    f = ref.glr_fwd(c, r, i, lam, lengths=n.tolist())
    off = ref.glr_fwd(1e-5 * mag, r, i, lam, lengths=n.tolist())
    # u, r and i themselves are fp32: a few half steps each, which the bounds' counts cover
    tol_h = 2 * (off["h_last"] + f["tol_h"])
    assert (np.abs(f64(state.h) - f["h_last"]) <= tol_h).all()
    for b, k in enumerate(n.tolist()):
        want = np.zeros((l.taps - 1, l.D))
        have = u[b, max(0, k - l.taps + 1):k]
        want[l.taps - 1 - len(have):] = have
        assert (np.abs(f64(state.conv[b]) - want) <= 8 * ref.U * np.abs(want)).all()
    v = (f["y"] * gate / (1 + np.exp(-gate))).reshape(B * L, l.D)
    top = np.abs(v).max(1)
    scale = top / 127
    units = v / np.where(scale > 0, scale, 1)[:, None]
    edge = np.abs(units - np.floor(units) - 0.5) < 1e-3
    w, sw = l.w_o[0].cpu().numpy().astype(np.float64), f64(l.w_o[1])
    want = (np.round(units) * scale[:, None]) @ (w * sw[:, None]).T
    slack = (edge * scale[:, None]) @ (np.abs(w) * sw[:, None]).T + 1e-4 * scale[:, None] * (np.abs(w).sum(1) * sw)
    assert (np.abs(f64(out).reshape(B * L, E) - want) <= slack + 1e-30).all()


def test_tokens_go_on_from_a_prompt():
    l = layer()
    B, L, E, T = 2, 70, 48, 5
    g = torch.Generator(device="cuda").manual_seed(6)
    x, res = (torch.randn(B, L, E, device="cuda", generator=g) for _ in range(2))
    n = torch.tensor([L - T, 2], dtype=torch.int32, device="cuda")
    _, _, whole = l.prompt(x, res, lengths=n + T)
    _, _, state = l.prompt(x, res, lengths=n)
    rows = torch.arange(B, device="cuda")
    for t in range(T):
        out, total = l.token(x[rows, n.long() + t], res[rows, n.long() + t], state)
        assert torch.isfinite(out).all()
        assert torch.equal(total, x[rows, n.long() + t] + res[rows, n.long() + t])
    # a row's codes do not depend on the rows beside it, and neither do its products
    assert torch.equal(state.conv, whole.conv)
    # both states are fp32 within the recurrence's and the convolution's share of the same fp64 one
    q, s, _ = seq.rmsnorm_q8(x.view(B * L, E), l.norm, residual=res.view(B * L, E))
    u, gates = (f64(seq.matmul_q8(q, s, *w, out_dtype=torch.float32)).reshape(B, L, -1) for w in (l.w_u, l.w_g))
    c, mag = conv64(u, l)
    r, i = gates[..., :l.D], gates[..., l.D:2 * l.D]
    f = ref.glr_fwd(c, r, i, f64(l.lam), lengths=(n + T).tolist())
    off = ref.glr_fwd(1e-5 * mag, r, i, f64(l.lam), lengths=(n + T).tolist())
    for s in (state, whole):
        assert (np.abs(f64(s.h) - f["h_last"]) <= off["h_last"] + f["tol_h"]).all()


def test_prompt_clamps_lengths():
    """Lengths below 0 and past L are 0 and L, for the convolution's window as for the recurrence."""
    l = layer()
    B, L, E = 4, 70, 48
    g = torch.Generator(device="cuda").manual_seed(8)
    x, res = (torch.randn(B, L, E, device="cuda", generator=g) for _ in range(2))
    n = torch.tensor([-5, L + 1, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    out, total, state = l.prompt(x, res, lengths=n)
    want = l.prompt(x, res, lengths=n.clamp(0, L))
    assert torch.equal(out, want[0]) and torch.equal(total, want[1])
    assert torch.equal(state.conv, want[2].conv) and torch.equal(state.h, want[2].h)


def test_mixer_gradients():
    """Each step's gradients from what the step before it gave, in fp64."""
    B, L, D, taps = 2, 90, 24, 4
    g = torch.Generator(device="cuda").manual_seed(7)
    u, r, i, dy = (torch.randn(B, L, D, device="cuda", generator=g) for _ in range(4))
    w, b = torch.randn(D, taps, device="cuda", generator=g), torch.randn(D, device="cuda", generator=g)
    l = layer(D=D)
    lengths = torch.tensor([90, 33], dtype=torch.int32, device="cuda")
    y, last, kept = recurrent.mixer_fwd(u, r, i, w, b, l.lam, lengths=lengths)
    du, dr, di, dw, db, dlam, dh0 = recurrent.mixer_bwd(dy, kept)
    c = kept[1]
    want = ref.glr_bwd(f64(dy), f64(c), f64(r), f64(i), f64(l.lam), lengths=lengths.tolist())
    for name, v in (("dr", dr), ("di", di), ("dlam", dlam), ("dh0", dh0)):
        assert (np.abs(f64(v) - want[name]) <= want["tol_" + name] + np.abs(want[name]) * 2 * ref.U).all(), name
    dc = torch.zeros(B, L + taps - 1, 1, D, device="cuda")
    seq.glr_bwd(dy, c, r, i, l.lam, kept[6], lengths=lengths, dx=dc[:, :L, 0])
    got = f64(dc[:, :L, 0])
    assert (np.abs(got - want["dx"]) <= want["tol_dx"] + np.abs(want["dx"]) * 2 * ref.U).all()
    args = (D, (1, 1), (taps - 1, 0), (1, 1))
    dw64, scale = oracle.conv_bwd_weight(f64(u).reshape(B, L, 1, D), f64(dc), D, (taps, 1), *args[1:])
    assert (np.abs(f64(dw).reshape(dw64.shape) - dw64) <= 1e-5 * scale).all()
    du64, scale = oracle.conv_bwd_data(f64(dc), f64(w).reshape(D, taps, 1, 1), D, (L, 1), *args[1:])
    assert (np.abs(f64(du).reshape(du64.shape) - du64) <= 1e-5 * scale).all()
    assert (np.abs(f64(db) - got.sum((0, 1))) <= 64 * ref.U * np.abs(got).sum((0, 1))).all()


def test_command_runs(capsys):
    recurrent.main(["--batch", "2", "--length", "96", "--dim", "64", "--width", "48", "--tokens", "3"])
    assert "prompt of 2 x 96 tokens" in capsys.readouterr().out
