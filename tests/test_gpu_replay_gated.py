"""The replayed training step of a gated block: the operators together, as a
program uses them, against float64 autograd of the same block with the same
masks, and what the replay finds."""
import pytest

import block_reference as ref
from bit_exact_matrix_amd import replay
from test_gpu_parity import say, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


def rms(torch, x, w, eps=1e-5):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * w


@pytest.mark.parametrize("dtype,sizes,drop", [("bf16", (300, 96, 260), 0.1),
                                              ("fp16", (64, 256, 512), 0.0),
                                              ("fp16", (33, 72, 200), 0.3),
                                              ("bf16", (1, 64, 128), 0.1)])
def test_step_against_autograd(torch_dev, dtype, sizes, drop):
    """E4M3 keeps values to within 2^-4; uniform errors of that size are off by
    2^-4 / sqrt(3) in the mean (0.036).  A gradient passes up to four such places
    (the checkpoints of h, g, u and a) and the product of two of them (g and u):
    0.18 with all of one sign.  The outputs see 16-bit roundings only: of r, h, a
    (once more after its mask), y, and their own, 2^-8 each at most, through a
    product of two projections (which counts h's twice)."""
    torch, dev = torch_dev
    rows, dim, hidden = sizes
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    p, x, branch, dr, dh = replay.make_gated(*sizes, dt, 3, dev)
    seed = 2 ** 40 + 7
    say("replayed gated step", dtype, sizes, drop)
    r2, h2, saved = replay.gated_forward(x, branch, p, drop, seed)
    dx, dbranch, grads = replay.gated_backward(dr, dh, saved, p, drop, seed)
    leaf = [t.double().requires_grad_() for t in (x, branch, *p)]
    lx, lb, nw, wg, wu, wd, gate, pw, qw = leaf
    inside, behind = (ref.mask(rows, n, drop, seed, o, dev) if drop else 1.0
                      for n, o in ((hidden, 0), (dim, 1)))
    r = lx + lb
    h = rms(torch, r, nw)
    y = (torch.nn.functional.silu(h @ wg) * (h @ wu) * inside) @ wd
    want_r = r + gate * (rms(torch, y, pw) * behind)
    want_h = rms(torch, want_r, qw)
    ((want_r * dr.double()).sum() + (want_h * dh.double()).sum()).backward()
    for got, want in ((r2, want_r.detach()), (h2, want_h.detach())):
        assert float((got.double() - want).norm() / want.norm()) < 7 * 2.0 ** -8
    for got, t in zip((dx, dbranch, *grads), leaf):
        assert got.shape == t.grad.shape
        assert float((got.double() - t.grad).norm() / t.grad.norm()) < 0.18


def test_findings(torch_dev):
    """The step repeats bit for bit.  Both products are within K 2^-23 of the
    exact sums of |terms| (K = 512, terms of one size: below 32 times the result),
    and the activation and the product of the two add their errors, with slopes
    of at most 1.1."""
    for model in ("hopper", "ampere"):
        say("replay of the gated block", model)
        found = replay.replay_gated(257, 512, 384, "bf16", model, seed=5)
        assert found["repeats"]
        assert 0 < found["emulated_relative_difference"] < 2.1 * 32 * 512 * 2.0 ** -23
        assert found["saved_bytes"] * 1.9 < found["whole_bytes"] and found["mask_bytes"] == 0


def test_another_mask_is_found(torch_dev, monkeypatch):
    """A backward pass whose mask is not the forward pass's (another offset, in
    one of the two runs)."""
    calls = [0]
    dropout = replay.blk.dropout

    def other(x, p, seed, offset, *args, **kw):
        calls[0] += 1
        return dropout(x, p, seed, offset + (calls[0] == 5), *args, **kw)

    say("replay of the gated block, another mask")
    monkeypatch.setattr(replay.blk, "dropout", other)
    assert not replay.replay_gated(65, 128, 256, dropout=0.2)["repeats"]


def test_emulated_rows_are_of_the_steps_products(torch_dev, monkeypatch):
    """A product that is wrong at the step's own number of rows only."""
    gated, rows = replay.blk.gated_linear, 257

    def wrong(x, *args, **kw):
        y, kept = gated(x, *args, **kw)
        return (y + 1 if x.shape[0] == rows else y), kept

    say("replay of the gated block, planted product")
    fine = replay.replay_gated(rows, 512, 384, seed=5)
    monkeypatch.setattr(replay.blk, "gated_linear", wrong)
    found = replay.replay_gated(rows, 512, 384, seed=5)
    assert fine["emulated_relative_difference"] < 1e-4
    assert found["emulated_relative_difference"] > 0.1


def test_the_step_in_a_captured_graph(torch_dev):
    """Captured once and replayed on new inputs and another seed on the device,
    each replay against the eager step."""
    torch, dev = torch_dev
    p, x, branch, dr, dh = replay.make_gated(96, 128, 320, torch.bfloat16, 1, dev)
    seed = torch.tensor([3, 4], dtype=torch.int64, device=dev)

    def step():
        # one mask's numbers serve both places here: a seed on the device has
        # its offset beside it
        blk = replay.blk
        before, behind = replay._ends(p)
        r, h, stats = blk.residual_norm(x, branch, before, pre="rms", dropout=0.1, seed=seed)
        a, kept = blk.gated_linear(h, p.w_gate, p.w_up, keep="checkpoint")
        a = blk.dropout(a, 0.1, seed)
        grads = blk.gated_linear_backward(blk.dropout_backward(a, 0.1, seed), h, p.w_gate, p.w_up,
                                          kept)
        back = blk.residual_norm_backward(dr, grads[0], r, branch, before, stats, pre="rms",
                                          dropout=0.1, seed=seed)
        return [r, h, a, *grads, *back[:2], back[2].pre_weight]

    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(replay.make_gated(96, 128, 320, torch.bfloat16, 50 + i, dev)[1])
        seed.copy_(torch.tensor([i, 100 + i]))
        say("gated step, graph replay", i)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_a_negative_seed(torch_dev):
    """As the plain block's replay takes it."""
    say("replay of the gated block, negative seed")
    found = [replay.replay(64, 128, 256, seed=-1), replay.replay_gated(64, 128, 256, seed=-1)]
    assert all(f["repeats"] for f in found)
