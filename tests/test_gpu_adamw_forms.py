"""The forms that AdamW's step takes by its hyperparameters, types and lists,
where one ends and the next begins, against the plain fp32 form."""
import numpy as np
import pytest

import adamw_common as A
import test_gpu_adamw as T
from test_gpu_adamw import dev, host

pytestmark = pytest.mark.gpu

F = np.float32
U = A.U


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(scope="module")
def oa():
    from communication_compressed_distributed_02_amd import ob_adamw
    return ob_adamw


def one_step(oa, m, v, g, b1, eps, lr=1.0):
    """A first step with 8-bit states from parameters of 0 and the moments'
    nearest codes: (x, m's codes and exponents) of the library and of the plain
    form, which continues from the decoded codes in fp32, one rounding per
    operation."""
    import torch
    n = m.size
    x = torch.zeros(n, device="cuda")
    opt = oa.AdamW([x], state_bits=8, betas=(b1, 0.999), eps=eps)
    opt.set("m", torch.from_numpy(m).cuda(), 0)
    opt.set("v", torch.from_numpy(v).cuda(), 0)
    m, v = A.decode_m(*A.encode_m(m)), A.decode_v(*A.encode_v(v, 1 << 19))
    assert A.same(host(opt.get("m", 0)), m) and A.same(host(opt.get("v", 0)), v)
    opt.step([dev(g)], lr)
    b1, eps = F(b1), F(eps)
    m = (b1 * m) + ((F(1) - b1) * g)
    v = (A.B2 * v) + (A.OB2 * (g * g))
    rbc2 = F(1.0 / np.sqrt(1.0 - float(A.B2)))
    rate = F(lr / (1.0 - float(b1)))
    want = -(rate * (m / ((np.sqrt(v) * rbc2) + eps)))
    view = opt.views()
    got = (host(x), view["m"].view(torch.uint8)[:n].cpu().numpy(),
           view["m_exp"][:n // 256].cpu().numpy())
    assert opt.check_guards() == -1
    return got, (want, *A.encode_m(m))


@pytest.mark.parametrize("b1", [0.0, 2.0 ** -8, 1.37 * 2.0 ** -9, 1.37 * 2.0 ** -20, 2.0 ** -70])
def test_moments_near_the_least_exponent_under_a_small_beta1(oa, b1):
    """First moments of 2^-111 to 2^-110, the least that the short form takes:
    b1 times their scale of 2^-118 is a normal number down to b1 = 2^-8.  Then,
    as for every group beside 8-bit moments, x is within 14 half steps of the
    update (here all of x; one more for the final rounding)."""
    r = np.random.RandomState(40)
    n = 4096
    m = (r.uniform(1.0, 2.0, n) * r.choice((-1, 1), n) * 2.0 ** -111).astype(F)
    v = np.full(n, 2.0 ** -60, F)
    for g in (np.zeros(n, F), (r.randn(n) * 2.0 ** -118).astype(F)):
        (x, codes, exps), (want, c, e) = one_step(oa, m, v, g, b1, 1e-8)
        least = np.abs(want[want != 0]).min() if want.any() else 1.0
        assert least > 2.0 ** -120 or b1 < 2.0 ** -60
        bad = np.abs(x.astype(np.float64) - want) > 15 * U * np.abs(want)
        assert not bad.any(), (b1, x[bad][:3], want[bad][:3])
        assert np.array_equal(np.where(codes & 127, codes, 0), np.where(c & 127, c, 0))
        assert np.array_equal(exps, e)


@pytest.mark.parametrize("eps", [2.0 ** -30, 1.0, 2.0 ** 90, 2.0 ** 100, 2.0 ** 125, 1e38, 3e38])
def test_updates_under_a_large_eps(oa, eps):
    """The reciprocal of a denominator past 2^126 is below the normal numbers;
    the update that it is a factor of is not."""
    r = np.random.RandomState(41)
    n = 4096
    m, v = np.zeros(n, F), np.full(n, 1e20, F)
    g = (r.uniform(0.5, 1.0, n) * r.choice((-1, 1), n) * 1e15).astype(F)
    (x, codes, exps), (want, c, e) = one_step(oa, m, v, g, 0.9, eps)
    assert np.abs(want).min() > 2.0 ** -100
    bad = np.abs(x.astype(np.float64) - want) > 15 * U * np.abs(want)
    assert not bad.any(), (eps, x[bad][:3], want[bad][:3])
    assert np.array_equal(codes, c) and np.array_equal(exps, e)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("bits,stochastic", [(32, False), (32, True), (8, False)])
def test_bfloat16_parameters_without_copies_under_float32_gradients(oa, bits, stochastic, many):
    """Ragged, unaligned, in one launch and in several, as the other kinds."""
    T.test_steps_equal_the_plain_form(oa, "bf16", "f32", bits, False, stochastic, many)


@pytest.mark.parametrize("g,big", [("f32", 17090 * 4096 + 1234), ("bf16", 32001 * 4096 + 77)])
def test_lists_past_every_round_and_launch(oa, g, big):
    """Lists so long that a block of the norm takes several chunks, not equally
    many (more than 2048 of them in a launch), forwards and, in front of a step,
    backwards, the fold a second round (more than 2048 partial sums), and a step
    two launches (more than 2^14 chunks) beside those of its tensors.  The gradients are small whole numbers, so S is exact
    in 64 bits whatever the order, and a chunk left out or taken twice shows;
    every element of m and v is compared, and the parameters around the places
    where launches and rounds meet."""
    import math

    import torch
    sizes = [1 + 61 * i % 9001 for i in range(500)]
    sizes[7], sizes[490] = big, 3 * 4096 + 1
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[g]
    gen = torch.Generator(device="cuda").manual_seed(44)
    gs = [torch.randint(-3, 4, (n,), device="cuda", generator=gen).to(dt) for n in sizes]
    xs = [torch.randn(n, device="cuda", generator=gen).mul_(0.1) for n in sizes]
    total = sum(int(a.to(torch.int32).square_().sum(dtype=torch.int64)) for a in gs)
    assert total < 1 << 53
    norm, s = oa.GradNorm(gs).grad_norm(gs)
    assert float(s) == total and float(norm) == F(math.sqrt(total))
    chunks = [-(-n // 4096) for n in sizes]
    launch = sum(chunks[:240])  # the first 240 tensors' chunks, in equal launches
    parts = -(-launch // (1 << 14))
    assert parts > 1 and len(sizes) > 480 and launch % 2048
    marks = [0, 2048, 4096] + [k * -(-launch // parts) for k in range(1, parts)]
    spots = {big - 300}
    for c in marks:
        at = 4096 * (c - sum(chunks[:7]))  # where chunk c lies in the big tensor
        spots.update(min(max(at + k * 4096 - 300, 0), big - 300) for k in (-1, 0, 1))
    pieces = {a: host(xs[7][a:a + 600]) for a in sorted(spots)}
    whole = {i: host(xs[i]) for i in (0, 3, 6, 8, 239, 240, 241, 479, 480, 490, 499)}
    opt = oa.AdamW(xs, grad_dtype=dt)
    got = opt.step(gs, 1e-2, 0.1, max_norm=1.0)
    assert float(got) == F(math.sqrt(total))
    gscale = float(F(1.0 / math.sqrt(total)))
    ob1, ob2 = float(A.OB1), float(A.OB2)
    view = opt.views()
    for i, a in enumerate(gs):
        at, n = opt.offsets[i], sizes[i]
        scaled = a.float() * gscale
        assert torch.equal(view["m"][at:at + n], scaled * ob1), i
        assert torch.equal(view["v"][at:at + n], (scaled * scaled) * ob2), i
        del scaled
    rows = [(a, xs[7][a:a + 600], gs[7][a:a + 600], p) for a, p in pieces.items()]
    rows += [(i, xs[i], gs[i], p) for i, p in whole.items()]
    for where, x, a, p in rows:
        zeros = np.zeros(p.size, F)
        want = A.step32(p, zeros, zeros, host(a), 1, 1e-2, 0.1, gscale)[0]
        assert A.same(host(x), want), where
    assert opt.check_guards() == -1 and opt.steps == (1, 0)
