"""The orthogonalised update against Newton-Schulz in 64 bits: shapes, spectra, types,
strides, scales from subnormal to overflowing squares, special values."""
import pytest
import torch

import dispatch_grouped_gemm_gb300 as hmm
from tests import open_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"

# wide, tall and square; one element; sizes around the tiles (256), the chunks (32) and
# the vectors (8); results that no tensor map can describe (odd N)
SHAPES = [(1, 1, 1), (1, 1, 40), (2, 40, 1), (3, 7, 5), (2, 16, 16), (1, 33, 100), (2, 128, 250),
          (1, 255, 257), (1, 256, 256), (2, 300, 70), (1, 513, 264), (2, 264, 513), (1, 520, 1040),
          (1, 1100, 600)]


def gradient(shape, spectrum="mixed", seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, device=DEV, dtype=torch.float64)

    B, M, N = shape
    if spectrum == "noise":
        return normal(B, M, N)
    r = max(1, min(M, N) // 16)
    low = normal(B, M, r) @ normal(B, r, N)
    if spectrum == "low rank":
        return low
    if spectrum == "decaying":
        k = min(M, N)
        return normal(B, M, k) * torch.logspace(0, -4, k, device=DEV, dtype=torch.float64) \
            @ normal(B, k, N)
    return low * (0.5 / r ** 0.5) + normal(B, M, N)


def check(g, got, **kw):
    """The kernels round where the model does, with other sums in fp32: other roundings
    of the same sizes, so that their error against 64 bits is the model's up to chance
    (a quarter for the norm, more for few elements), plus the result's own rounding (half
    a step at most) and the fp32 sums (2^-20).  One element may be off by four times the
    model's worst in so few draws.

    Below 64 elements the model's few roundings can all be small by luck (with one
    element its error was 1.2e-4 where another rounding of A gives 1.1e-3), so an
    arithmetic bound stands for them.  One step takes a singular value x to x B',
    B' = a + b s + c s^2, s = x^2.  Rounding hi (twice in A) and A changes s by at most 3
    half steps, 3 * 2^-11 s, and so x B' by 3 * 2^-11 x s |b + 2 c s|; rounding B' changes
    it by 2^-11 x |B'|.  With the usual coefficients x stays below 1.203 (the largest
    image of [0, 1.203]), where x s |b + 2 c s| <= 1.92 and x |B'| <= 1.203: 2^-11 (3 * 1.92
    + 1.203) = 7 * 2^-11 a step.  The step before reaches the result times
    |d(x B') / dx| <= 4 there, and one before that times less than 16; steps whose errors
    all add up are far from what can happen by chance, so two steps' worth, 7 (1 + 4) *
    2^-11 = 35 * 2^-11, is what a mistake has to exceed."""
    want = ref.orthogonalize(g, **kw)
    model = ref.orthogonalize(g, rounded=True, **kw)
    half = torch.finfo(got.dtype).eps / 2
    for w, m, y in zip(want.reshape(-1, *g.shape[-2:]), model.reshape(-1, *g.shape[-2:]),
                       got.double().reshape(-1, *g.shape[-2:])):
        assert bool(torch.isfinite(y).all())
        if w.numel() < 64:
            size = abs(kw.get("scale", 1.0))
            assert bool(((y - w).abs() <= 35 * 2.0 ** -11 * size + half * w.abs()).all())
            continue
        norm, rms = w.norm(), w.square().mean().sqrt()
        e = (m - w).norm()
        # (few elements: chance counts for more)
        few = 1.25 + 8.0 / max(1, w.numel()) ** 0.5
        assert (y - w).norm() <= few * e + (half + 2.0 ** -20) * norm
        worst = (m - w).abs().max()
        assert bool(((y - w).abs() <= 4 * worst + half * w.abs() + 2.0 ** -18 * rms
                     + torch.finfo(got.dtype).tiny).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype):
    g = gradient(shape).to(dtype)
    got = hmm.orthogonalize(g)
    assert got.dtype == (torch.float16 if dtype == torch.float16 else torch.bfloat16)
    assert got.shape == g.shape
    check(g, got)


@pytest.mark.parametrize("spectrum", ["noise", "mixed", "low rank", "decaying"])
@pytest.mark.parametrize("shape", [(2, 300, 520), (1, 520, 300), (1, 512, 512)])
def test_spectra(shape, spectrum):
    g = gradient(shape, spectrum).float()
    got = hmm.orthogonalize(g)
    check(g, got)
    # what the precision is for: within half a percent of 64 bits for every spectrum
    want = ref.orthogonalize(g)
    assert (got.double() - want).norm() <= 0.005 * want.norm()


@pytest.mark.parametrize("kw", [
    dict(steps=1), dict(steps=2, scale=0.2), dict(steps=8), dict(steps=5, scale=-3.0),
    dict(steps=12, coefficients=(1.5, -0.5, 0.0)), dict(steps=3, coefficients=(2.0, -1.5, 0.5)),
    dict(steps=3, coefficients=((4.0, -6.0, 2.8), (3.4, -4.7, 2.0), (1.9, -1.3, 0.4))),
    dict(steps=2, eps=0.5)])
def test_parameters(kw):
    g = gradient((2, 100, 136)).float()
    check(g, hmm.orthogonalize(g, **kw), **kw)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [128, 129])
def test_result_types(out, N):
    g = gradient((2, 72, N)).float()
    got = hmm.orthogonalize(g, out_dtype=out)
    assert got.dtype == out
    check(g, got)


@pytest.mark.parametrize("dtype,size", [(torch.float32, 1e-42), (torch.float32, 1e-30),
                                        (torch.float32, 1e-15), (torch.float32, 1e25),
                                        (torch.float32, 3e37), (torch.bfloat16, 1e-38),
                                        (torch.bfloat16, 1e36), (torch.float16, 1e-5),
                                        (torch.float16, 6e4)])
def test_sizes_of_elements(dtype, size):
    """Elements whose squares overflow or vanish in fp32."""
    g = gradient((1, 60, 80))
    g = (g / g.abs().max() * size).to(dtype)
    check(g, hmm.orthogonalize(g, eps=0.0), eps=0.0)


def test_mixed_sizes_in_one_norm():
    g = gradient((3, 50, 64)).float()
    g[0, :25] *= 1e-25
    g[1, :25] *= 1e25
    g[2, 10:20] = 0
    check(g, hmm.orthogonalize(g), eps=1e-7)


def test_special_values():
    """Zeros give zeros; an infinity or a NaN stays in its matrix."""
    g = gradient((4, 40, 72)).to(torch.bfloat16)
    clean = hmm.orthogonalize(g)
    g[0] = 0
    g[1, 3, 5] = float("nan")
    g[2, 7, 1] = float("inf")
    got = hmm.orthogonalize(g)
    assert not bool(got[0].any())
    assert bool(torch.isnan(got[1]).any()) and bool(torch.isnan(got[2]).any())
    assert torch.equal(got[3], clean[3])
    assert not bool(hmm.orthogonalize(torch.zeros((2, 5, 6), device=DEV), eps=0.0).any())


def test_strides():
    big = gradient((6, 90, 200)).to(torch.bfloat16)
    for g in (big[:, :60, :100], big[::2, 1:61, 3:103], big[:, :80, :60].transpose(1, 2),
              big[0], big[0, :, :64].T, big[:1, :60, :100].expand(4, 60, 100),
              big[:, :, ::2], big.view(2, 3, 90, 200), big.view(2, 3, 90, 200)[:, :2]):
        got = hmm.orthogonalize(g)
        assert got.shape == g.shape and got.is_contiguous()
        assert torch.equal(got, hmm.orthogonalize(g.clone(memory_format=torch.contiguous_format)))


def test_a_matrix_does_not_depend_on_its_stack():
    g = gradient((5, 280, 300)).to(torch.bfloat16)
    got = hmm.orthogonalize(g)
    for i in range(5):
        assert torch.equal(got[i], hmm.orthogonalize(g[i]))


def test_empty():
    assert hmm.orthogonalize(torch.empty((0, 8, 8), device=DEV)).shape == (0, 8, 8)
    assert hmm.orthogonalize(torch.empty((3, 0, 8), device=DEV)).shape == (3, 0, 8)


def test_many_tiles():
    g = gradient((3, 1408, 2048)).to(torch.bfloat16)
    check(g, hmm.orthogonalize(g))


def test_refused_while_differentiating():
    g = gradient((1, 8, 8)).float().requires_grad_()
    with pytest.raises(RuntimeError, match="no backward"):
        hmm.orthogonalize(g)
    with torch.no_grad():
        hmm.orthogonalize(g)


@pytest.mark.parametrize("spectrum", ["mixed", "low rank", "decaying"])
@pytest.mark.parametrize("shape", [(4, 128, 250), (3, 300, 200), (2, 65, 1000), (1, 520, 768),
                                   (40, 264, 270)], ids=str)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32], ids=str)
def test_fp16_results_are_exact_to_their_rounding(shape, dtype, spectrum):
    """Of a result in fp16 its own rounding shows, half a step, 2^-11 of each value at
    most, or half of 2^-24, and the fp32 sums: an MMA adds to an accumulator that loses
    2^-24 of the largest partial sum, 3 * 1000 / 16 of them in a sum at most, 2^-16, some
    four times the result where terms cancel; fifteen products with a sensitivity of at
    most 4 to the end add up to 2^-12 at most if all err alike.  (Operands in 11 bits
    would be off by 2^-10.)"""
    g = gradient(shape, spectrum).to(dtype)
    got = hmm.orthogonalize(g, out_dtype=torch.float16)
    want = ref.orthogonalize(g)
    assert got.dtype == torch.float16
    err = (got.double() - want).flatten(1).norm(dim=1)
    least = 2.0 ** -25 * (shape[1] * shape[2]) ** 0.5
    assert bool((err <= (2.0 ** -11 + 2.0 ** -12) * want.flatten(1).norm(dim=1) + least).all())
    assert torch.equal(got, hmm.orthogonalize(g, out_dtype=torch.float16))


@pytest.mark.parametrize("shape,steps", [((3, 279, 28), 4), ((36, 1000, 19), 5), ((2, 64, 300), 5),
                                         ((5, 420, 387), 6), ((2, 512, 600), 8),
                                         ((1, 600, 900), 6)], ids=str)
def test_small_matrices_and_many_steps(shape, steps):
    """bf16 results of small matrices, and of many steps, are exact to their rounding
    too: half a step, 2^-8 of each value at most, and the fp32 sums' part of the test
    above, 2^-12 times the steps over five."""
    g = gradient(shape).to(torch.bfloat16)
    got = hmm.orthogonalize(g, steps=steps).double()
    want = ref.orthogonalize(g, steps=steps)
    # (spread evenly, a rounding is half a step / sqrt(3) of values up to twice as large as
    # their power of two: below 2^-8 / sqrt(3) over a whole matrix but for chance)
    bound = 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -12 * steps / 5
    assert bool(((got - want).flatten(1).norm(dim=1) <= bound * want.flatten(1).norm(dim=1)).all())
