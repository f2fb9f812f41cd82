"""Attention over the 4-bit cache against 64 bits, by the error of each head (or of 64 channels of one) relative to its
norm, where values differ in size between channels, positions and pages."""
import numpy as np
import pytest
import torch

import decoder_only_b200 as lb
import _serving as ref
from test_gpu_serving import FUTURE, MANY, _attend, _attend_case, _scales

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _errors(c, got, width):
    """|got - want| / |want| of every `width` channels of every row, by norms; [rows, H * hd / width]."""
    want, _ = ref.attention(c["q64"], c["pool"], c["table"], c["lens"], c["cu"], c["n_kv"], False)
    want = want.reshape(len(want), -1, width)
    off = got.double().cpu().numpy().reshape(want.shape) - want
    size = np.linalg.norm(want, axis=-1)
    none = size == 0                                          # rows that see nothing
    assert not off[none].any()
    return np.where(none, 0.0, np.linalg.norm(off, axis=-1) / np.where(none, 1.0, size))


# Roundings to nearest of independent numbers, each 2^-p at the most and a 1.7th of it on average: the output to bf16
# (p = 9), 2^-9.8; weights times steps or keys, values and weights in fp16 (p = 12), which against codes that all have
# one sign weigh twice, 2^-10.8 a time: below 2^-9 together.  Twice that for one head of thousands.
FINE = 2.0 ** -8
# A page whose values differ widely in size takes weights and values in bf16 (p = 9 each, about the size of the output's own
# rounding): below 2^-8.5 together, doubled again
WIDE = 2.0 ** -7.5


@pytest.mark.parametrize("H,n_kv,hd,lens,new", [s for s in FUTURE if s[2] == 128] + [(16, 8, 128, [700, 260], [130, 256])])
@pytest.mark.parametrize("group", [0, 1])
@pytest.mark.parametrize("power", [-60, -36, -24, -12, 12, 24, 36])
@pytest.mark.parametrize("where", ["all", "some", "first page", "last page"])
def test_attention_with_64_channels_of_the_values_of_another_size(H, n_kv, hd, lens, new, group, power, where):
    """One group's values 2^power times as large: at every position, at a third of them, in the first or the last page."""
    c = _attend_case(H + hd + 2, lens, new, H, n_kv, hd, BF16)
    zs, put = _scales(c, hd)
    rng = np.random.default_rng(3)
    for b, length in enumerate(lens):
        for pos in range(length):
            if {"all": True, "some": rng.random() < 0.33, "first page": pos < 128, "last page": pos // 128 == (length - 1) // 128}[where]:
                zs[c["table"][b, pos // 128], :, pos % 128 // 32, 1, pos % 32, group] += (power << 7) & 0xffff
    put()
    e = _errors(c, _attend(c), 64)
    print("largest error", e.max())
    assert e.max() <= WIDE, e.max()
    assert lb.op_last_error() == 0


@pytest.mark.parametrize("H,n_kv,hd,lens,new", [s for s in FUTURE if s[2] == 128])
@pytest.mark.parametrize("group", [0, 1])
@pytest.mark.parametrize("power", [-60, 30, 100, None])
def test_attention_rows_do_not_depend_on_64_channels_that_come_after_them(H, n_kv, hd, lens, new, group, power):
    c = _attend_case(H + hd + 3, lens, new, H, n_kv, hd, BF16)
    zs, put = _scales(c, hd)
    for b, length in enumerate(lens):
        for pos in (length - 2, length - 1):
            at = zs[c["table"][b, pos // 128], :, pos % 128 // 32, 1, pos % 32, group]
            at[:] = 0x7fc0 if power is None else at + ((power << 7) & 0xffff)
    put()
    out = _attend(c)
    rows = np.concatenate([np.arange(c["cu"][b], c["cu"][b + 1] - 2) for b in range(len(lens))])
    e = _errors(c, out, 64)[rows]
    print("largest error", e.max())
    assert e.max() <= WIDE, e.max()


@pytest.mark.parametrize("H,n_kv,hd,lens,new", MANY + [
    (32, 8, 128, [2014, 1381, 777], [384, 448, 1]), (14, 2, 64, [129, 900], [129, 200]), (5, 1, 64, [400], [400]),
    (4, 4, 128, [40, 300, 1], [9, 6, 1]), (9, 3, 64, [70, 33, 500], [8, 3, 1]),           # few columns
    (8, 1, 128, [9001], [1]), (12, 12, 64, [33, 2000, 5], [1, 1, 1]),
])
def test_attention_error_relative_to_each_head(H, n_kv, hd, lens, new):
    c = _attend_case(H + hd + 4, lens, new, H, n_kv, hd, BF16, poison=True, strided=True)
    e = _errors(c, _attend(c), hd)
    print("largest error", e.max(), "rms", np.sqrt((e ** 2).mean()))
    assert e.max() <= FINE, e.max()
    assert lb.op_last_error() == 0


@pytest.mark.parametrize("H,n_kv,hd,lens,new", [(32, 4, 128, [100, 300], [100, 80]), (16, 16, 64, [700, 300], [250, 300]),
                                                (8, 2, 128, [300, 40], [9, 3]), (6, 6, 64, [513], [1])])
@pytest.mark.parametrize("sharp", [4.0, 16.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_error_of_peaked_softmax(H, n_kv, hd, lens, new, sharp, dtype):
    """Queries that are keys of their sequence, so that a few positions hold nearly all of the weight and the running
    maximum moves.  A score's error moves a weight in proportion: scores of sharp * sqrt(hd) and less, of which fp16
    (many columns: queries and keys, 2^-12 each and independent over hd channels) gets 2^-11.5 / 1.7 / sqrt(hd) of |q||k|
    wrong, under sharp * 2^-12 of 1; fp32's products 2^-20."""
    rng = np.random.default_rng(9)
    c = _attend_case(H + hd + 5, lens, new, H, n_kv, hd, dtype)
    K, _, _, _ = ref.unpack(c["pool"], hd)
    G = H // n_kv
    q = np.zeros((len(c["q"]), H, hd))
    for b, (length, n) in enumerate(zip(lens, new)):
        for i in range(n):
            for h in range(H):
                pos = rng.integers(0, length - n + i + 1)
                k = K[c["table"][b, pos // 128], h // G, pos % 128]
                q[c["cu"][b] + i, h] = sharp * np.sqrt(hd) / np.linalg.norm(k) ** 2 * k
    t = torch.from_numpy(q).to(dtype)
    c["q"], c["q64"] = t.cuda(), t.double().numpy()
    e = _errors(c, _attend(c), hd)
    print("largest error", e.max(), "rms", np.sqrt((e ** 2).mean()))
    assert e.max() <= (FINE + sharp * 2.0 ** -11 if dtype == BF16 else 2.0 ** -18), e.max()


@pytest.mark.parametrize("H,n_kv,hd,lens,new", [(32, 4, 128, [100, 700], [100, 300]), (16, 16, 64, [700, 300], [250, 300]),
                                                (8, 2, 128, [300, 40], [9, 3]), (6, 6, 64, [513], [1])])
@pytest.mark.parametrize("bits", [12, 20])
def test_attention_beside_a_position_that_takes_the_weight_and_gives_nothing(H, n_kv, hd, lens, new, bits):
    """A first position of zero values whose score is about `bits` above the others' in base 2: what is left of the weights
    makes the result.  fp16 rounds what is below 2^-14 to multiples of 2^-24, by 2^-25 at the most: with many columns 2^7
    times a weight, so 2^-32 of its value; with few 2^5 times a weight and more times its step over the largest step, so
    2^-30 of the largest step, and that for up to 15 of them, below 2^-29 of the largest value (|z| is half of 15 steps
    here).  Scores vary by several bits (rows of few positions may have weights of 2^-30 alone), so that is added to the
    relative bound: 2^-29 of the largest value for each position, in the norm of hd channels."""
    c = _attend_case(H + hd + 6, lens, new, H, n_kv, hd, BF16)
    q = c["q"].abs()
    c["q"], c["q64"] = q, q.double().cpu().numpy()
    zs, put = _scales(c, hd)
    # |q| has 0.8 hd as its sum: a key of z everywhere has a score of 0.8 sqrt(hd) z log2(e) in base 2
    z = torch.tensor(bits / (0.8 * hd ** 0.5 * 1.4427), dtype=BF16).view(torch.int16).item()
    for b in range(len(lens)):
        at = zs[c["table"][b, 0], :, 0, :, 0]             # [heads, keys or values, groups, (z, s)]
        at[:, 0] = [z, 0]
        at[:, 1] = 0
    put()
    e = _errors(c, _attend(c), hd)
    first = [c["cu"][b] for b in range(len(lens)) if new[b] == lens[b]]      # rows that see that position alone: zeros
    assert not e[first].any()
    print("largest error", e.max(), "rms", np.sqrt((e ** 2).mean()))
    want, _ = ref.attention(c["q64"], c["pool"], c["table"], c["lens"], c["cu"], n_kv, False)
    _, V, _, _ = ref.unpack(c["pool"], hd)
    size = np.linalg.norm(want.reshape(e.shape + (hd,)), axis=-1)
    seen = np.concatenate([length - n + 1 + np.arange(n) for length, n in zip(lens, new)])[:, None]
    bound = WIDE * size + seen * 2.0 ** -29 * np.abs(V).max() * hd ** 0.5
    assert np.all(e * size <= bound), (e * size / bound).max()
