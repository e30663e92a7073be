"""8-bit scores over the whole range of the scales (bytes 1 to 254), against 64 bits (tolerances as in
test_gpu_residual)."""
import pytest
import torch

from differentiable_gaussian_splat_amd import labels as L

from .test_gpu_labels import BF16, DEV, F32, IDS, TYPES, U, empty, gen, half_step, randn, within
from .test_gpu_residual import E8, Q8, check_scores, dequantize

pytestmark = pytest.mark.gpu

# few rows straight from memory, one wave's and several waves' depth; tiles of each size
SIZES = [(1, 128, 40), (3, 1024, 1000), (16, 384, 33_000), (40, 640, 300), (300, 8192, 70), (517, 4224, 1003),
         (1500, 384, 1500), (4000, 640, 4090), (8192, 512, 5120)]


def codes(g, n, cols):
    """Every finite e4m3 value."""
    q = torch.randint(0, 256, (n, cols), generator=g, device=DEV).to(torch.uint8)
    q[(q & 127) == 127] = 1
    return q.view(Q8)


def bytes_of(s, n, cols):
    """Scales of the given bytes [n, cols / 128], padded."""
    pad = -(cols // 128) % 4
    return torch.nn.functional.pad(s.to(torch.uint8), (0, pad), value=127).view(E8)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("byte", [1, 2, 9, 15, 16, 239, 240, 246, 247, 253])
def test_ends(byte, dtype):
    """Rows at one end against words at the other, products of ordinary size."""
    g = gen(byte)
    for n, cols, vocab in ((5, 640, 200), (500, 640, 3000)):
        near = lambda k, at: bytes_of((at + torch.randint(-2, 3, (k, cols // 128), generator=g, device=DEV))
                                      .clamp(1, 254), k, cols)
        rows, words = (codes(g, n, cols), near(n, byte)), (codes(g, vocab, cols), near(vocab, 254 - byte))
        check_scores(rows, words, dtype)
        check_scores(words, rows, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("swap", [False, True], ids=["rows", "words"])
@pytest.mark.parametrize("n,cols,vocab", SIZES)
def test_every_scale_beside_every_other(n, cols, vocab, swap, dtype):
    """Scales drawn for each row and block, of either operand from the whole range and of the other from its low part.
    Compared where float32 holds the sum and all that counts in it: magnitudes of 2^-90 (terms below float32's numbers,
    65536 of 2^-126, are 2^-20 of it, and less than the tolerance) to 2^126."""
    g = gen(n + cols + vocab)
    draw = lambda k, end: bytes_of(torch.randint(1, end, (k, cols // 128), generator=g, device=DEV), k, cols)
    rows = codes(g, n, cols), draw(n, 96 if swap else 255)
    words = codes(g, vocab, cols), draw(vocab, 255 if swap else 96)
    out = empty(n, vocab, dtype=dtype)
    L.gs_label_scores_q8(*rows, *words, out)
    a, b = dequantize(*rows), dequantize(*words)
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    tol = mag * (2 * cols * U) + ref.abs() * half_step(dtype)
    if dtype is BF16:
        tol = tol + 2.0 ** -10 * (a.abs().reshape(n, -1, 8).amax(2) @ b.abs().reshape(vocab, -1, 8).amax(2).t())
    here = (mag >= 2.0 ** -90) & (mag <= 2.0 ** 126)
    assert here.float().mean() > 0.1
    within("scores", torch.where(here, out.double(), 0.0), torch.where(here, ref, 0.0), tol)


@pytest.mark.parametrize("shift", [0, 110, 111, 112, 115, 119, -119])
@pytest.mark.parametrize("n,cols,vocab", SIZES)
def test_float32_sums_of_whole_numbers_are_exact(n, cols, vocab, shift):
    """Values of -2 to 2, and in the first two columns of every eight 64 * 64, which cancels; scales of 1, 2 and 4 times
    2^shift against those times 2^-shift. Every sum is a whole number below 2^24, in whatever order it is made: what a
    unit cuts off beside large products, or takes from another's scale, shows."""
    g = gen(n * 3 + cols + vocab)
    sides = []
    for k, at, second in ((n, shift, 64), (vocab, -shift, -64)):
        q = torch.randint(-2, 3, (k, cols), generator=g, device=DEV).float()
        q[:, 0::8], q[:, 1::8] = 64, second
        s = torch.randint(127, 130, (k, cols // 128), generator=g, device=DEV) + at
        sides.append((q.to(Q8), bytes_of(s, k, cols)))
    out = empty(n, vocab)
    L.gs_label_scores_q8(*sides[0], *sides[1], out)
    assert torch.equal(out.double(), dequantize(*sides[0]) @ dequantize(*sides[1]).t())


def test_quantised_ends():
    """The scales that the quantiser itself gives the largest and the smallest float32 rows."""
    g = gen(4)
    big = torch.full((40, 300), 3.4e38, device=DEV) * torch.where(randn(g, 40, 300) > 0, 1.0, -1.0)
    small = randn(g, 70, 300) * 2.0 ** -124
    for rows, words in ((big, small), (small, big)):
        check_scores(L.quantize_q8(rows), L.quantize_q8(words), F32)
        check_scores(L.quantize_q8(rows), L.quantize_q8(words), BF16)


@pytest.mark.parametrize("share", [0.003, 0.1])
@pytest.mark.parametrize("side", [0, 1], ids=["rows", "words"])
@pytest.mark.parametrize("n,cols,vocab", [(40, 640, 3000), (300, 1024, 300), (4000, 640, 4090), (9001, 128, 8003),
                                          (8192, 512, 6144), (8192, 1024, 8192)])
def test_far_and_near_tiles_in_turn(n, cols, vocab, side, share):
    """Some rows (or words) of whole numbers are 2^-115 of the others: tiles with and without them follow one another in
    a block, and each score is exact."""
    g = gen(n + cols + vocab + side)
    sides = []
    for k, which in ((n, 0), (vocab, 1)):
        q = torch.randint(-2, 3, (k, cols), generator=g, device=DEV).float().to(Q8)
        s = torch.randint(127, 130, (k, cols // 128), generator=g, device=DEV)
        if which == side:
            s = s - 115 * (torch.rand((k, 1), generator=g, device=DEV) < share)
        sides.append((q, bytes_of(s, k, cols)))
    want = dequantize(*sides[0]) @ dequantize(*sides[1]).t()
    for _ in range(3):
        out = empty(n, vocab)
        L.gs_label_scores_q8(*sides[0], *sides[1], out)
        assert torch.equal(out.double(), want)
