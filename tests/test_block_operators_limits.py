"""The block operators at their limits: calls without groups, and calls that one
launch does not hold."""
import pytest
import torch

import bit_exact_fp8_amd as fw
from bit_exact_fp8_amd import block_operators
from test_block_operators import E8, blocks, c_grouped, c_weight_grad, check_grouped, dev, exact_codes, spans, spread  # noqa: F401
from test_operators import BF, E4, SF, f64, note, rand, rng


# ---- no group at all ---------------------------------------------------------
@pytest.mark.parametrize("kw", [dict(K=250, lda=250, ldw=250), dict(a=17), dict(lda=257), dict(a=None), dict(lda=0), dict(od=2, K=250)])
def test_no_groups_need_no_workspace(kw):
    """With the size that the query gives such a call is not refused for it, whatever a's
    rows look like, which are not read: the pointer's alignment is all that is left to refuse."""
    lib = block_operators._lib()
    assert lib.emu_grouped_block_scaled_mm_workspace(1000, 0, 300, kw.get("K", 256), kw.get("od", 0), 0, 0) == 0
    assert c_grouped(E=0, ws=8, wsb=0, **kw) == 1
    assert b"workspace is not 16-byte aligned" in lib.emu_last_error_message()


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(1, 250), (65, 256), (100, 250), (900, 250), (900, 256)])
@pytest.mark.parametrize("out", [BF, SF])
def test_no_groups(dev, T, K, out):  # noqa: F811
    note(f"grouped product {T}x300x{K} of no groups")
    a = torch.zeros(T, K + 3, dtype=torch.uint8, device=dev)[:, 1:1 + K].view(E4)
    args = (a, torch.empty(0, 300, K, dtype=E4, device=dev).transpose(1, 2), torch.zeros(T, blocks(K), device=dev).to(E8),
            torch.empty(0, blocks(300), blocks(K), device=dev).to(E8).transpose(1, 2), torch.empty(0, dtype=torch.int32, device=dev))
    y = fw.grouped_block_scaled_mm(*args, out_dtype=out)
    assert y.shape == (T, 300) and not y.any()
    given = torch.full((T, 300), 7.0, dtype=out, device=dev)
    assert (fw.grouped_block_scaled_mm(*args, out_dtype=out, out=given) == 7).all()
    # without operands, through the C ABI, and with more workspace than is asked for
    given.fill_(7.0)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize(dev)
    status = c_grouped(a=None, w=None, sa=None, sw=None, ends=None, E=0, M=T, K=K, lda=K, ldw=K, od=2 if out == SF else 0, out=given.data_ptr(),
                       ws=ws.data_ptr(), wsb=ws.numel())
    torch.cuda.synchronize(dev)
    assert status == 0 and not given.any()


# ---- more than one launch holds -------------------------------------------------
def alike(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def repeated(t, T):
    """`t` over and over, T rows."""
    return t.repeat(-(-T // len(t)), 1)[:T]


@pytest.mark.gpu
def test_more_blocks_than_a_launch(dev):  # noqa: F811
    """2^29 rows of one value, of which a grid of 2^32 threads would be one launch:
    those of a small call over and over, at every border between launches too."""
    T, period = 2 ** 29 + 33, 2 ** 20 + 7
    gen = torch.Generator(device=dev).manual_seed(5)
    gate, up, g = (torch.randn(period, 1, device=dev, generator=gen).to(BF) for _ in range(3))
    want, want_h = fw.block_quant(gate), fw.swiglu_block_quant(gate, up, keep=True)
    want_d = fw.swiglu_block_backward(g, want_h.kept, want_h.kept_scale)

    def check(got, want):
        for y, w in zip(got, want):
            assert len(y) == T
            for r in range(0, T, period):
                assert alike(y[r:r + period], w[:min(period, T - r)]), r

    note(f"block codes of {T} rows")
    gate, up, g = (repeated(t, T) for t in (gate, up, g))
    check(fw.block_quant(gate), want)
    note(f"gated activation of {T} rows")
    h = fw.swiglu_block_quant(gate, up, keep=True)
    check(h, want_h)
    note(f"gated activation's gradient of {T} rows")
    check([fw.swiglu_block_backward(g, h.kept, h.kept_scale)], [want_d])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(2 ** 18, 2 ** 16 + 4), (2 ** 16 + 3, 2 ** 17 + 5)])
def test_more_outputs_than_a_launch(dev, M, N):  # noqa: F811
    """Without K the bias is every row, also where there are more than 2^34 outputs or slices of them."""
    note(f"block product {M}x{N}x0")
    b = torch.randn(N, device=dev, generator=torch.Generator(device=dev).manual_seed(7)).to(BF)
    z = lambda *s: torch.empty(*s, dtype=E4, device=dev)  # noqa: E731
    y = fw.block_scaled_mm(z(M, 0), z(N, 0).t(), torch.empty(M, 0, device=dev), torch.empty(blocks(N), 0, device=dev).t(), bias=b)
    assert y.shape == (M, N)
    for r in range(0, M, 4096):
        assert (y[r:r + 4096] == b).all(), r


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("ends,T,K,pad", [([1, 2], 3, 48, (0, 0)), ([0, 3], 3, 48, (3, 5)), ([2], 5, 33, (0, 0)), ([70, 290], 300, 48, (0, 0)),
                                          ([130, 280], 300, 33, (0, 0)), ([200, 200], 300, 32, (0, 5))])
def test_grouped_columns_of_several_launches(dev, ends, T, K, pad, given):  # noqa: F811
    """More columns than a launch takes: of few rows, of tiles, and of operands laid out anew for each launch."""
    check_grouped(dev, ends, T, 2 ** 17 + 130, K, exact=True, given=given, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("T,K", [(300, 16), (300, 33), (2000, 16)])
def test_many_groups_of_several_launches(dev, T, K, given):  # noqa: F811
    """As many groups as there may be, of which a launch takes a few hundred columns."""
    E, N = 65536, 514
    note(f"grouped product {T}x{N}x{K} of {E} groups given={given}")
    a, sa, av = exact_codes(rng(T + K), T, K, 1, E4, E8)
    gen = torch.Generator(device=dev).manual_seed(T)
    w = torch.randint(-1, 2, (E, N, K), device=dev, generator=gen, dtype=torch.int8).to(BF).to(E4)
    sw = torch.randint(127, 129, (E, blocks(N), blocks(K)), device=dev, generator=gen, dtype=torch.uint8).view(E8)
    ends = torch.randint(0, T - 9, (E,), generator=rng(K)).sort().values
    ends[-1] = T - 9
    o = torch.full((T, N + 3), 7.0, dtype=BF, device=dev)[:, 2:2 + N] if given else None
    y = fw.grouped_block_scaled_mm(a.to(dev), w.transpose(1, 2), sa.to(dev), sw.transpose(1, 2), ends.to(dev), out=o)
    want = torch.full((T, N), 7.0 if given else 0.0, dtype=f64, device=dev)
    av = av.to(dev)
    for e, (first, end) in enumerate(spans(ends.tolist(), T)):
        if end > first:
            wv = w[e].to(f64) * spread(sw[e].float().to(f64), N, K, 128)
            want[first:end] = av[first:end] @ wv.t().contiguous()
    assert torch.equal(y, want.to(BF))
    if given:
        assert (o._base[:, :2] == 7).all() and (o._base[:, 2 + N:] == 7).all()


# ---- outputs that meet themselves ------------------------------------------------
@pytest.mark.parametrize("kw,fine", [(dict(os=64 * 256), True), (dict(os=64 * 256 - 1), False), (dict(os=1), False), (dict(os=255), False),
                                     (dict(os=300, ldo=900), True), (dict(os=256, ldo=768), True), (dict(os=256, ldo=767), False),
                                     (dict(os=300, ldo=855), False), (dict(os=63 * 300 + 256, ldo=300), True),
                                     (dict(os=63 * 300 + 255, ldo=300), False), (dict(N=1, os=256, ldo=256), True),
                                     (dict(N=1, os=255, ldo=256), False)])
def test_weight_grad_outputs_apart(kw, fine):
    """Matrices one after the other or row by row among each other, but not over each other
    (all that is left to refuse then is the workspace's alignment)."""
    assert c_weight_grad(ends=16, E=3, ws=8, **kw) == 1
    text = block_operators._lib().emu_last_error_message()
    assert (b"workspace is not 16-byte aligned" in text) == fine and (b"overlap" in text) != fine


@pytest.mark.gpu
def test_weight_grad_of_interleaved_outputs(dev):  # noqa: F811
    """Experts' matrices row by row beside each other, as [N, E, K] holds them; over each other they are refused."""
    T, N, K, ends = 90, 40, 130, torch.tensor([20, 50, 90], device=dev)
    c, s, _ = exact_codes(rng(1), T, K, 1, E4, E8)
    g = torch.randint(-2, 3, (T, N), generator=rng(2)).to(BF).to(dev)
    out = torch.empty(N, 3, K, dtype=BF, device=dev).transpose(0, 1)
    want = fw.block_weight_grad(g, c.to(dev), s.to(dev), ends)
    assert torch.equal(fw.block_weight_grad(g, c.to(dev), s.to(dev), ends, out=out), want)
    with pytest.raises(fw.EmuError):
        fw.block_weight_grad(g, c.to(dev), s.to(dev), ends, out=out._base.as_strided((3, N, K), (N * K - 1, K, 1)))


# ---- sums over a token's choices --------------------------------------------------
@pytest.mark.gpu
def test_expert_step_adds_choices_in_their_order(dev):  # noqa: F811
    """A token's experts' outputs, and its inputs' gradients, are added in the order
    of its choices: the same bits on every run."""
    from bit_exact_fp8_amd import expert_step as es
    T, n, hidden, E, c = 700, 256, 128, 12, 5
    gen = rng(4)
    x, grad, share = rand(gen, T, n).to(dev), rand(gen, T, n).to(dev), torch.rand(T, c, generator=gen).to(dev)
    up, down = es.project(rand(gen, E, 2 * hidden, n, std=n ** -0.5).to(dev)), es.project(rand(gen, E, n, hidden, std=0.1).to(dev))
    choice = torch.randint(0, E, (T, c), generator=gen).to(dev)  # (the same expert twice too)
    with torch.no_grad():
        out, kept = es.forward(x, up, down, choice, share)
        g = es.backward(grad, kept, up, down, share)

        def joined(rows):
            """Of rows by expert: each token's, added one after the other."""
            at = torch.empty_like(kept.order)
            at[kept.order] = torch.arange(T * c, device=dev)
            rows = rows[at].view(T, c, n)
            y = rows[:, 0]
            for j in range(1, c):
                y = y + rows[:, j]
            return y

        y = es._product(kept.h.codes, kept.h.scale, down.codes, down.scale, kept.ends, SF)
        assert torch.equal(out, joined(y * share.reshape(-1)[kept.order, None]))
        rows = grad[kept.order // c] * share.reshape(-1)[kept.order, None]
        codes, scale = fw.block_quant(rows)
        grad_h = es._product(codes, scale, down.turned, down.turned_scale, kept.ends, SF)
        codes, scale = fw.block_quant(fw.swiglu_block_backward(grad_h, kept.h.kept, kept.h.kept_scale))
        assert torch.equal(g.x, joined(es._product(codes, scale, up.turned, up.turned_scale, kept.ends, SF)))


@pytest.mark.gpu
@pytest.mark.parametrize("T,c", [(5, 0), (0, 2)])
def test_expert_step_without_rows(dev, T, c):  # noqa: F811
    """Tokens of no expert, and no tokens: zeros, and no gradient."""
    from bit_exact_fp8_amd import expert_step as es
    up, down = es.project(rand(rng(1), 3, 256, 128).to(dev)), es.project(rand(rng(2), 3, 128, 128).to(dev))
    x, choice, share = torch.ones(T, 128, device=dev), torch.zeros(T, c, dtype=torch.int64, device=dev), torch.zeros(T, c, device=dev)
    out, kept = es.forward(x, up, down, choice, share)
    g = es.backward(x, kept, up, down, share)
    assert out.shape == g.x.shape == (T, 128) and not out.any() and not g.x.any() and not g.up.any() and not g.down.any()
