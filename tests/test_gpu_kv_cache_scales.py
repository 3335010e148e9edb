"""Attention over E4M3 caches whose rows have very different scales: a row's
result is that of the stored values, whatever the magnitudes of its neighbours in
the cache, hidden ones among them.

Bounds (kv_reference.py has the rest).  P is FP16: half a step is 2^-11 relative
(torch.finfo(torch.float16).eps / 2).
Its smallest step is 2^-36 of the row's largest weight (times the value's size) in
the step kernel.  In the chunk kernel it is 2^-32 of the weight at the reference,
which counts the largest scale of 32 values, up to 2^8 times a value's own: 2^-24;
beyond that every value's own scale counts.  Values of zeros count like their
neighbours.  An exponent is the difference of numbers up to 2^8,
rounded twice in FP32 (2^-17 each, times ln 2): 2^-16 of a weight."""
import numpy as np
import pytest
import torch

import kv_reference as R
from bit_attention_gb300 import kv_cache as KV
from bit_attention_gb300 import sage_fp4 as S

pytestmark = pytest.mark.gpu

# a few rows a sequence and head (the step kernel), many (the chunk kernel)
FEW, MANY = ([3, 1], [200, 64]), ([150, 96], [230, 200])


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def filled(k, v, q_lens, kv_lens, H, D, page=16, seed=0):
    """A batch whose sequences' tokens are the rows k, v [all tokens, H, D]."""
    b = R.Batch("e4m3", H, D, page, q_lens, kv_lens, seed=seed, fill=False)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(kv_lens)]).astype(np.int32)).cuda()
    KV.append(b.cache, bf16(k), bf16(v), cu, b.kv_len, b.block_table)
    return b


def check(b, q, many, **kw):
    o, lse = KV.attention(q, b.cache, *b.args(), return_lse=True, **kw)
    assert b.cache.get_status() == S.OK
    R.check_attention(b, q, o, lse, p_step=2.0 ** -11, least=2.0 ** (-24 if many else -36), slack=2.0 ** -16, zeros=many, **kw)


def one_hot(n, D, size):
    """[n, 1, D]: row j is size[j] at channel j mod D."""
    x = np.zeros((n, 1, D))
    x[np.arange(n), 0, np.arange(n) % D] = size
    return x


def aimed(b, D, keys, size):
    """Queries [T, heads, D] that hit the channel of keys[t, h] with `size`."""
    q = np.zeros((b.T, keys.shape[1], D))
    t, h = np.indices(keys.shape)
    q[t, h, keys % D] = size
    return bf16(q)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [8, 24, 40, 100])
@pytest.mark.parametrize("lens", [FEW, MANY])
def test_the_weight_on_values_far_smaller_than_their_neighbours(D, most, lens):
    # values of 2^0 .. 2^-most within every 32 keys, the softmax on one channel's keys
    rng = np.random.default_rng(most + D)
    n = sum(lens[1])
    v = rng.standard_normal((n, 1, D)) * 2.0 ** -rng.integers(0, most + 1, (n, 1, 1))
    v[::9] = 0.0
    b = filled(one_hot(n, D, np.full(n, 8.0)), v, *lens, 1, D)
    keys = rng.integers(0, D, (b.T, 4))
    check(b, aimed(b, D, keys, 100.0 * D ** 0.5 / 8), lens is MANY)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("most", [8, 24, 40, 100])
@pytest.mark.parametrize("lens", [FEW, MANY])
def test_keys_far_smaller_than_their_neighbours(D, most, lens):
    # keys of 2^0 .. 2^-most within every 32, queries whose size makes up for it
    rng = np.random.default_rng(most + D + 1)
    n = sum(lens[1])
    down = rng.integers(0, most + 1, D)[np.arange(n) % D]  # the same of all keys of a channel
    b = filled(one_hot(n, D, 8.0 * 2.0 ** -down), rng.standard_normal((n, 1, D)), *lens, 1, D)
    keys = rng.integers(0, D, (b.T, 4))
    size = np.zeros(D)
    size[np.arange(n) % D] = 2.0 ** down
    check(b, aimed(b, D, keys, 5.0 * D ** 0.5 / 8 * size[keys]), lens is MANY)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("up", [6, 20, 30, 60])
@pytest.mark.parametrize("lens", [([3, 2], [200, 64]), MANY])
@pytest.mark.parametrize("side", ["k", "v"])
def test_hidden_tokens_of_any_size_change_nothing(D, up, lens, side):
    # tokens 2^up times larger: the last two of a sequence, which the others do not
    # see, and one that the window hides from all of them
    rng = np.random.default_rng(up + D)
    n = sum(lens[1])
    q = None
    for window in (None, 20):
        k, v = rng.standard_normal((2, n, 2, D))
        end = 0
        for nq, m in zip(*lens):
            end += m
            (k if side == "k" else v)[end - 2:end] *= 2.0 ** up
            if window:
                (k if side == "k" else v)[end - nq - 21] *= 2.0 ** up
        b = filled(k, v, *lens, 2, D, page=64)
        q = bf16(rng.standard_normal((b.T, 8, D))) if q is None else q
        check(b, q, lens is MANY, window=window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("spread", [3, 8, 16, 30])
@pytest.mark.parametrize("lens", [FEW, MANY])
def test_rows_of_all_sizes(D, spread, lens):
    # keys and values scaled by 2^-spread .. 1 at random, rows of zeros among them
    rng = np.random.default_rng(spread + D)
    n = sum(lens[1])
    k, v = rng.standard_normal((2, n, 2, D)) * 2.0 ** -rng.uniform(0, spread, (2, n, 2, 1))
    k[::11], v[5::7] = 0.0, 0.0
    b = filled(k, v, *lens, 2, D, page=32)
    q = bf16(3.0 * rng.standard_normal((b.T, 6, D)))
    for kw in (dict(), dict(causal=False), dict(window=70, scale=0.3)):
        check(b, q, lens is MANY, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [([2, 1], [5000, 1500]), ([130, 70], [5000, 1500])])
@pytest.mark.parametrize("sizes", [(0, -70, 0, -100), (-60, 60, -60, 0), (-90, 40, 0, 20), (110, -60, 110, 0)])
def test_stretches_of_tokens_of_very_different_sizes(D, lens, sizes):
    # values of one size for hundreds of tokens, in turn: shares that are joined,
    # references that move by more than FP32's exponents; a stretch of zeros between
    rng = np.random.default_rng(D)
    n = sum(lens[1])
    k, v = rng.standard_normal((2, n, 1, D))
    for i in range(0, n, 300):
        v[i:i + 300] *= 2.0 ** sizes[i // 300 % 4]
        v[i + 40:i + 100] = 0.0
    b = filled(k, v, *lens, 1, D, page=64)
    check(b, bf16(rng.standard_normal((b.T, 4, D))), lens[0][0] > 4)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [([2, 1], [3000, 700]), ([130, 70], [3000, 700])])
@pytest.mark.parametrize("high,low", [(100, -20), (90, -60), (30, -70)])
def test_stretches_of_mixed_and_of_small_values(D, lens, high, low):
    # 300 tokens whose values are 2^high and 2^(high - 12) in turn, then 300 of 2^low
    rng = np.random.default_rng(D + high)
    n = sum(lens[1])
    k, v = rng.standard_normal((2, n, 1, D))
    i = np.arange(n)
    v *= 2.0 ** np.where(i // 300 % 2 == 0, high - 12.0 * (i % 2), low)[:, None, None]
    b = filled(k, v, *lens, 1, D, page=32)
    check(b, bf16(rng.standard_normal((b.T, 4, D))), lens[0][0] > 4)


@pytest.mark.parametrize("lens", [([2], [20000]), ([140], [20000])])
@pytest.mark.parametrize("halves", [(90, -60), (-60, 90), (0, -95)])
def test_halves_of_a_long_sequence_of_very_different_sizes(lens, halves):
    # shares that see one size alone and are joined: the weights of both count
    rng = np.random.default_rng(7)
    n = lens[1][0]
    k, v = rng.standard_normal((2, n, 1, 64))
    v *= 2.0 ** np.where(np.arange(n) < n // 2, *map(float, halves))[:, None, None]
    b = filled(k, v, *lens, 1, 64, page=64)
    check(b, bf16(rng.standard_normal((b.T, 4, 64))), lens[0][0] > 4)


@pytest.mark.parametrize("lens", [FEW, MANY])
def test_rows_of_zeros_and_next_to_zero(lens):
    # magnitudes down to bf16's smallest, where the scale's byte stops at its least
    rng = np.random.default_rng(3)
    n = sum(lens[1])
    k, v = rng.standard_normal((2, n, 1, 64))
    v[::3], v[1::3] = 0.0, v[1::3] * 2.0 ** -130
    k[2::5] *= 2.0 ** -120
    b = filled(k, v, *lens, 1, 64)
    check(b, bf16(rng.standard_normal((b.T, 4, 64))), lens is MANY)
    b = filled(k, 0.0 * v, *lens, 1, 64)
    check(b, bf16(rng.standard_normal((b.T, 4, 64))), lens is MANY)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [17, 32, 33])
def test_rows_next_to_the_border_of_the_kernels(fmt, D, G):
    # one token under 17, 32 and 33 query heads over thousands of cached tokens:
    # two row tiles of the step kernel in several shares, and the chunk kernel (whose
    # values' scales are within 2^2 here)
    b = R.Batch(fmt, 2, D, 64, [1, 1, 1], [6000, 300, 2500], seed=G)
    q = bf16(2.0 * b.rng.standard_normal((b.T, 2 * G, D)))
    for window in (None, 2000):
        o, lse = KV.attention(q, b.cache, *b.args(), window=window, return_lse=True)
        assert b.cache.get_status() == S.OK
        R.check_attention(b, q, o, lse, window=window, p_step=2.0 ** -11, least=2.0 ** (-36 if G <= 32 else -30))
