"""The paged cache on the GPU: rows written, read back and attended to, against
the plain 64-bit forms of kv_reference.py.  Stored codes and scales, and rows
read back, have to be exact; attention's bounds are derived there."""
import numpy as np
import pytest
import torch

import kv_reference as R
from bit_attention_gb300 import kv_cache as KV
from bit_attention_gb300 import sage_fp4 as S

pytestmark = pytest.mark.gpu

FORMATS = ("bf16", "e4m3", "nvfp4")


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


# ------------------------------------------------------------------ append, read
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,page,q_lens,kv_lens", [
    (1, 16, [1], [1]),
    (8, 64, [1, 1, 1], [1, 64, 65]),
    (3, 16, [2, 0, 5], [4, 3, 5]),
    (2, 16, [37, 1, 200], [50, 1, 333]),
    (5, 1024, [40], [1050]),
    (19, 32, [3], [40]),  # more heads than a warp takes
])
def test_append_stores_the_rule_and_nothing_else(fmt, D, H, page, q_lens, kv_lens):
    b = R.Batch(fmt, H, D, page, q_lens, kv_lens, seed=D + H, fill=False)
    c = b.cache
    before = [x.clone() for x in c.buffers[:-1]]
    x = b.rng.standard_normal((b.T, 2 * H, D)) * np.exp(3 * b.rng.standard_normal((b.T, 2 * H, 1)))
    x[::7, 0] = 0.0                      # rows of zeros
    x[1::7, :, :16] *= 1e-4              # groups that round to nothing in 4 bits
    x[2::5, :, 5] = 448.0 * 2.0 ** b.rng.integers(-6, 6)  # a largest magnitude at the border of a scale
    kv = bf16(x)
    KV.append(c, kv[:, :H], kv[:, H:], *b.args())
    torch.cuda.synchronize()
    assert c.get_status() == S.OK
    for w, part in (("k", kv[:, :H]), ("v", kv[:, H:])):
        codes, scales = getattr(c, w + "_codes"), getattr(c, w + "_scales")
        want = [t for t, n in zip(before, ("k", "v") if fmt == "bf16" else ("k", "v", "ks", "vs")) if n[0] == w]
        want = [t.cpu() for t in want]
        for s in range(b.B):
            page_, slot = (r[kv_lens[s] - q_lens[s]:] for r in b.rows(s))
            rows = part[b.cu[s]:b.cu[s + 1]].cpu()
            if fmt == "bf16":
                want[0][page_, :, slot] = rows
            else:
                wc, ws = R.store(R.f64(rows), fmt)
                want[0][page_, :, slot], want[1][page_, :, slot] = torch.from_numpy(wc), torch.from_numpy(ws)
        view = (lambda t: t.view(torch.int16)) if fmt == "bf16" else (lambda t: t)
        assert torch.equal(view(codes.cpu()), view(want[0])), w
        if fmt != "bf16":
            assert torch.equal(scales.cpu(), want[1]), w


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_takes_the_extremes_of_bf16(fmt):
    b = R.Batch(fmt, 1, 64, 16, [6], [6], fill=False)
    x = np.zeros((6, 2, 64))
    x[0, :, 0], x[1, :, 1], x[2, :, 2] = 3.3895e38, 2.0 ** -126, 2.0 ** -133
    x[3, :, :] = -3.3895e38
    x[4, :, 3], x[4, :, 4] = 1.0, -1e-30
    kv = bf16(x)
    KV.append(b.cache, kv[:, :1], kv[:, 1:], *b.args())
    k, v = KV.read(b.cache, b.kv_len, b.block_table, 6)
    for got, rows in ((k, kv[:, :1]), (v, kv[:, 1:])):
        if fmt == "bf16":
            assert torch.equal(got[0, 0], rows[:, 0])
        else:
            c, s = (torch.from_numpy(t) for t in R.store(R.f64(rows[:, 0]), fmt))
            assert np.array_equal(R.f64(got[0, 0]), R.values(c, s, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("D,H,page,kv_lens,N", [(64, 3, 16, [0, 1, 17, 100], 70), (128, 8, 64, [200, 64], 200),
                                               (128, 1, 32, [5], 1), (64, 2, 128, [129], 300)])
def test_read_returns_the_stored_values(fmt, layout, D, H, page, kv_lens, N):
    b = R.Batch(fmt, H, D, page, [0] * len(kv_lens), kv_lens, seed=N)
    wide = [torch.full((b.B, H, N, D + 8) if layout == "HND" else (b.B, N, H, D + 8), 7.0, dtype=torch.bfloat16,
                       device="cuda") for _ in range(2)]
    out = [x[..., :D] for x in wide]
    assert KV.read(b.cache, b.kv_len, b.block_table, N, layout=layout, out=out)[0] is out[0]
    assert b.cache.get_status() == S.OK
    for w, x, whole in zip("kv", out, wide):
        assert (whole[..., D:] == 7.0).all()
        x = x if layout == "HND" else x.transpose(1, 2)
        for s, n in enumerate(kv_lens):
            want = np.zeros((H, N, D))
            m = min(n, N)
            if m:
                want[:, :m] = b.dense(w, s)[:, :m]
            assert np.array_equal(R.f64(x[s]), want), (w, s)


def test_bad_indexes_are_recorded_and_left_out():
    b = R.Batch("e4m3", 2, 64, 16, [40, 3], [40, 50], seed=1)
    torch.cuda.synchronize()
    ok = [x.clone() for x in b.cache.buffers[:-1]]
    kv = bf16(b.rng.standard_normal((43, 4, 64)))
    for value in (-1, b.cache.num_pages, 2 ** 31 - 1, -2 ** 31):
        bad = b.block_table.clone()
        bad[0, 1] = value  # tokens 16..31 of sequence 0
        for x, y in zip(b.cache.buffers, ok):
            x.copy_(y)
        KV.append(b.cache, kv[:, :2], kv[:, 2:], b.cu_q, b.kv_len, bad)
        assert b.cache.get_status() == S.EINDEX and b.cache.get_status() == S.OK
        page = int(b.table[0, 1])
        assert torch.equal(b.cache.k_codes[page], ok[0][page]) and torch.equal(b.cache.v_scales[page], ok[3][page])
        k, v = KV.read(b.cache, b.kv_len, bad, 50)
        assert b.cache.get_status() == S.EINDEX
        assert (k[0, :, 16:32] == 0).all() and (v[0, :, 16:32] == 0).all() and (k[0, :, 32:40] != 0).any()
        q = bf16(b.rng.standard_normal((43, 4, 64)))
        o, lse = KV.attention(q, b.cache, b.cu_q, b.kv_len, bad, return_lse=True)
        assert b.cache.get_status() == S.EINDEX
        R.check_attention(b, q, o, lse, lost=[(0, j) for j in range(16, 32)])
    # lengths that the table cannot hold: the sequence counts as empty
    for n in (-1, b.block_table.shape[1] * 16 + 1, 2 ** 31 - 1):
        lens = b.kv_len.clone()
        lens[0] = n
        o = torch.full((43, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        q = bf16(b.rng.standard_normal((43, 4, 64)))
        KV.attention(q, b.cache, b.cu_q, lens, b.block_table, out=o)
        assert b.cache.get_status() == S.EINDEX
        assert (o[:40] == 0).all() and (o[40:] != 0).any()
        k, _ = KV.read(b.cache, lens, b.block_table, 50)
        assert b.cache.get_status() == S.EINDEX and (k[0] == 0).all() and (k[1] != 0).any()
    # rows past the packed tensors: the sequence has no new tokens
    for cu in ([0, 40, 44], [0, 50, 43], [-1, 40, 43]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o = torch.full((43, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
        KV.attention(q, b.cache, cu, b.kv_len, b.block_table, out=o)
        assert b.cache.get_status() == S.EINDEX
        KV.append(b.cache, kv[:, :2], kv[:, 2:], cu, b.kv_len, b.block_table)
        assert b.cache.get_status() == S.EINDEX


def test_tokens_before_the_first_position_and_rows_behind_the_last_are_left():
    # five new tokens of a sequence of three: the first two have no position;
    # rows 5.. of the packed tensors belong to nobody
    b = R.Batch("bf16", 2, 64, 16, [5], [3], fill=False)
    kv = bf16(b.rng.standard_normal((8, 4, 64)))
    KV.append(b.cache, kv[:, :2], kv[:, 2:], *b.args())
    page = int(b.table[0, 0])
    assert torch.equal(b.cache.k_codes[page, :, :3], kv[2:5, :2].transpose(0, 1))
    assert int(torch.isfinite(b.cache.k_codes).sum()) == 3 * 2 * 64
    q = bf16(b.rng.standard_normal((8, 2, 64)))
    out = torch.full((8, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    _, lse = KV.attention(q, b.cache, *b.args(), out=out, return_lse=True)
    R.check_attention(b, q, out, lse)
    assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all() and (out[5:] == 5.0).all()
    assert b.cache.get_status() == S.OK


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,G,page,q_lens,kv_lens", [
    (1, 1, 16, [1], [1]),
    (2, 4, 64, [1, 1, 1, 1], [1, 63, 128, 700]),          # single tokens
    (1, 7, 16, [1, 0, 1], [1000, 5, 0]),                  # one sequence has nothing new, one nothing cached
    (2, 3, 16, [2, 5, 1], [130, 5, 257]),                 # a few tokens each
    (1, 8, 32, [64], [64]),                               # a prompt
    (2, 2, 128, [130, 1, 300], [500, 400, 300]),          # chunks and a single token together
    (1, 20, 16, [3], [40]),                               # more heads a group than a row tile
    (3, 1, 64, [129], [1000]),
])
def test_attention_matches_the_plain_form(fmt, D, H, G, page, q_lens, kv_lens):
    b = R.Batch(fmt, H, D, page, q_lens, kv_lens, seed=H * 100 + G)
    q = bf16(2.0 * b.rng.standard_normal((b.T, H * G, D)))
    for causal, window, scale in ((True, None, None), (False, None, 0.2), (True, 50, None), (True, 1, None), (False, 77, None)):
        o, lse = KV.attention(q, b.cache, *b.args(), causal=causal, window=window, scale=scale, return_lse=True)
        assert b.cache.get_status() == S.OK
        R.check_attention(b, q, o, lse, causal=causal, window=window, scale=scale, label=f"causal={causal} window={window}")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 1, 1], [9000, 33, 2500], 4), ([300, 40], [5000, 3333], 2)])
def test_attention_over_long_caches(fmt, q_lens, kv_lens, G):
    b = R.Batch(fmt, 2, 128, 64, q_lens, kv_lens, seed=5)
    q = bf16(2.0 * b.rng.standard_normal((b.T, 2 * G, 128)))
    for window in (None, 3000):
        o, lse = KV.attention(q, b.cache, *b.args(), window=window, return_lse=True)
        assert b.cache.get_status() == S.OK
        R.check_attention(b, q, o, lse, window=window)


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [300]), ([150], [300])])
def test_large_scores_and_equal_scores(q_lens, kv_lens):
    # scores of several hundred (one key takes all), then queries of zeros (all alike)
    b = R.Batch("bf16", 1, 64, 16, q_lens, kv_lens, seed=8)
    for q in (bf16(200.0 * b.rng.standard_normal((b.T, 4, 64))), bf16(np.zeros((b.T, 4, 64)))):
        o, lse = KV.attention(q, b.cache, *b.args(), return_lse=True)
        R.check_attention(b, q, o, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [411, 90]), ([5, 1], [415, 33]), ([290, 7], [700, 400])])
def test_pages_that_a_window_hides_may_be_gone(fmt, D, page, q_lens, kv_lens):
    b = R.Batch(fmt, 2, D, page, q_lens, kv_lens, seed=13)
    q = bf16(b.rng.standard_normal((b.T, 6, D)))
    for window in (1, 40, 200):
        ref = KV.attention(q, b.cache, *b.args(), window=window, return_lse=True)
        R.check_attention(b, q, *ref, window=window)
        table = b.block_table.clone()
        for s, (nq, n) in enumerate(zip(q_lens, kv_lens)):
            table[s, :max(0, n - nq - window + 1) // page] = -7
        got = KV.attention(q, b.cache, b.cu_q, b.kv_len, table, window=window, return_lse=True)
        assert b.cache.get_status() == S.OK
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        # the last page of those still seen is not one of them
        for s in (0, 1):
            table[s, max(0, kv_lens[s] - q_lens[s] - window + 1) // page] = -7
            KV.attention(q, b.cache, b.cu_q, b.kv_len, table, window=window)
            assert b.cache.get_status() == S.EINDEX


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 5]), ([150, 1], [300, 5])])
def test_queries_of_zeros_and_next_to_zero_under_any_scale(fmt, q_lens, kv_lens):
    # their factors to scores underflow; masked keys stay out all the same
    b = R.Batch(fmt, 1, 128, 16, q_lens, kv_lens, seed=12)
    x = b.rng.standard_normal((b.T, 4, 128))
    x[:, 0], x[:, 1], x[:, 2] = 0.0, x[:, 1] * 2.0 ** -120, x[:, 2] * 2.0 ** -60
    q = bf16(x)
    for scale in (1e-9, 1e-30, 1e-38, None):
        for window in (None, 20):
            o, lse = KV.attention(q, b.cache, *b.args(), scale=scale, window=window, return_lse=True)
            R.check_attention(b, q, o, lse, scale=scale, window=window, label=f"scale={scale}")
    assert b.cache.get_status() == S.OK


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 2], [6, 40], 4), ([6], [6], 4), ([60, 2], [61, 300], 7)])
def test_weights_next_to_nothing_under_a_steep_softmax(fmt, D, q_lens, kv_lens, G):
    # where the leading key's value is a zero of its format, the result is made of
    # weights down to FP16's smallest
    b = R.Batch(fmt, 3, D, 32, q_lens, kv_lens, seed=27)
    q = bf16(2.0 * b.rng.standard_normal((b.T, 3 * G, D)))
    for scale in (0.5, 1.0):
        o, lse = KV.attention(q, b.cache, *b.args(), scale=scale, return_lse=True)
        R.check_attention(b, q, o, lse, scale=scale)
    assert b.cache.get_status() == S.OK


@pytest.mark.parametrize("q_lens,kv_lens,G", [([1, 1], [600, 31], 4), ([200, 3], [600, 31], 2)])
def test_attention_takes_strided_queries_and_outputs(q_lens, kv_lens, G):
    b = R.Batch("e4m3", 2, 64, 16, q_lens, kv_lens, seed=3)
    Hq = 2 * G
    packed = bf16(b.rng.standard_normal((b.T, Hq + 4, 64)))
    heads_first = bf16(b.rng.standard_normal((Hq, b.T, 64))).transpose(0, 1)
    for q in (packed[:, :Hq], packed[:, 2:2 + Hq], heads_first):
        ref = KV.attention(q.contiguous(), b.cache, *b.args())
        room = torch.full((Hq, b.T + 3, 72), 3.0, dtype=torch.bfloat16, device="cuda")
        out = room.transpose(0, 1)[:b.T, :, :64]
        KV.attention(q, b.cache, *b.args(), out=out)
        assert torch.equal(out, ref)
        assert (room[:, b.T:] == 3.0).all() and (room[..., 64:] == 3.0).all()


def test_outputs_of_shared_memory_and_other_misfits_are_refused():
    b = R.Batch("e4m3", 2, 64, 16, [3, 1], [20, 9])
    q = bf16(b.rng.standard_normal((4, 4, 64)))
    one = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    dense = torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")
    cu, n, table = b.args()
    for call in (lambda: KV.attention(q, b.cache, *b.args(), out=one.expand(4, 4, 64)),
                 lambda: KV.attention(q, b.cache, *b.args(), out=one[:, :1].expand(4, 4, 64)),
                 lambda: KV.attention(q, b.cache, *b.args(), out=q.as_strided((4, 4, 64), (256, 32, 1)).clone()[:3]),
                 lambda: KV.attention(q, b.cache, *b.args(), workspace=ws),
                 lambda: KV.attention(q, b.cache, *b.args(), workspace=q),
                 lambda: KV.attention(q, b.cache, *b.args(), window=0),
                 lambda: KV.attention(q, b.cache, *b.args(), scale=0.0),
                 lambda: KV.attention(q[:, :3], b.cache, *b.args()),
                 lambda: KV.attention(q.float(), b.cache, *b.args()),
                 lambda: KV.attention(q[..., ::2], b.cache, *b.args()),
                 lambda: KV.attention(q[..., 4:].contiguous(), b.cache, *b.args()),
                 lambda: KV.attention(q, b.cache, cu.long(), n, table),
                 lambda: KV.attention(q, b.cache, cu[:-1], n, table),
                 lambda: KV.attention(q, b.cache, cu, n, table[:1]),
                 lambda: KV.attention(q, b.cache, cu, n, table[:1].expand(2, -1)),
                 lambda: KV.attention(q, b.cache, cu, n, table.t().contiguous().t()),
                 lambda: KV.attention(q, b.cache, cu, n, table.cpu()),
                 lambda: KV.append(b.cache, kv, kv[:3], *b.args()),
                 lambda: KV.append(b.cache, q, q, *b.args()),
                 lambda: KV.append(b.cache, kv.view(-1)[4:260].view(2, 2, 64), kv[:2], *b.args()),
                 lambda: KV.read(b.cache, n, table, 8, out=(dense, dense[:1].expand(2, 2, 8, 64))),
                 lambda: KV.read(b.cache, n, table, 7, out=(dense, dense)),
                 lambda: KV.read(b.cache, n, table, -1),
                 lambda: KV.read(b.cache, n, table, 8, layout="NHHD")):
        with pytest.raises(S.SageFp4Error) as e:
            call()
        assert e.value.code == S.EINVAL
    assert b.cache.get_status() == S.OK


def test_empty_calls():
    b = R.Batch("bf16", 2, 64, 16, [0, 0], [5, 0])
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    KV.append(b.cache, e, e, *b.args())
    odd = e.as_strided((0, 2, 64), (0, 0, 0))  # no element, any strides
    KV.append(b.cache, odd, odd, *b.args())
    assert KV.attention(odd, b.cache, *b.args(), out=odd) is odd
    assert KV.attention(e, b.cache, *b.args()).shape == (0, 2, 64)
    k, _ = KV.read(b.cache, b.kv_len, b.block_table, 0)
    assert k.shape == (2, 2, 0, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 4.0)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    KV.attention(q, b.cache, one, none, b.block_table[:0], out=out)
    assert (out == 4.0).all() and b.cache.get_status() == S.OK


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_captured_step_follows_changing_lengths(fmt):
    # append + attention of one token a sequence, captured once, replayed as the
    # sequences grow over page borders; then against the eager calls
    b = R.Batch(fmt, 2, 64, 16, [1, 1, 1], [15, 100, 300], seed=9, spare=9)
    b.block_table[0, 1] = b.cache.num_pages and int(sorted(set(range(b.cache.num_pages)) - set(b.table[b.table >= 0]))[0])
    b.table[0, 1] = int(b.block_table[0, 1])
    kv, q = bf16(np.zeros((3, 4, 64))), bf16(np.zeros((3, 8, 64)))
    ws = torch.empty(KV.attention_workspace_bytes(b.cache, 3, 3, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty((3, 8, 64), dtype=torch.bfloat16, device="cuda")

    def step():
        KV.append(b.cache, kv[:, :2], kv[:, 2:], *b.args())
        KV.attention(q, b.cache, *b.args(), out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        if i:
            b.kv_len += torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
            b.kv_lens = [n + d for n, d in zip(b.kv_lens, (1, 0, 1))]
        kv.copy_(bf16(b.rng.standard_normal((3, 4, 64))))
        q.copy_(bf16(b.rng.standard_normal((3, 8, 64))))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        R.check_attention(b, q, out)
        ref = KV.attention(q, b.cache, *b.args())
        assert torch.equal(ref, out)
    assert b.cache.get_status() == S.OK


def test_calls_on_another_stream():
    b = R.Batch("e4m3", 2, 128, 64, [4, 1], [400, 900], seed=2)
    q = bf16(b.rng.standard_normal((5, 8, 128)))
    ref = KV.attention(q, b.cache, *b.args())
    rk, rv = KV.read(b.cache, b.kv_len, b.block_table, 900)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda._sleep(2_000_000)
        q2 = q * 1.0  # made on the current stream just before
        o = KV.attention(q2, b.cache, *b.args(), stream=side)
        k, v = KV.read(b.cache, b.kv_len, b.block_table, 900, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, ref) and torch.equal(k, rk) and torch.equal(v, rv)
    assert b.cache.get_status() == S.OK


@pytest.mark.parametrize("q_lens,kv_lens", [([1] * 5, [3000, 10, 777, 1500, 64]), ([400, 30], [2000, 900])])
def test_repeated_runs_are_bit_identical(q_lens, kv_lens):
    b = R.Batch("nvfp4", 2, 128, 16, q_lens, kv_lens, seed=4)
    q = bf16(b.rng.standard_normal((b.T, 8, 128)))
    runs = [KV.attention(q, b.cache, *b.args(), return_lse=True) for _ in range(4)]
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])


def test_a_prompt_in_chunks_is_the_prompt_at_once():
    # stored and attended to in chunks of odd sizes: each chunk against the plain form
    b = R.Batch("nvfp4", 2, 64, 16, [0], [333], seed=6, fill=False)
    kv = bf16(b.rng.standard_normal((333, 4, 64)))
    q = bf16(b.rng.standard_normal((333, 6, 64)))
    at = 0
    for n in (100, 1, 31, 128, 73):
        b.q_lens, b.kv_lens, b.T = [n], [at + n], n
        b.cu = np.array([0, n])
        b.cu_q, b.kv_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [at + n]))
        part = slice(at, at + n)
        KV.append(b.cache, kv[part, :2], kv[part, 2:], *b.args())
        o, lse = KV.attention(q[part], b.cache, *b.args(), return_lse=True)
        R.check_attention(b, q[part], o, lse)
        at += n


def test_sequences_read_back_feed_the_fp4_attention():
    # bf16 rows come back as they went in, so the dense FP4 attention gives the same bits
    H, N, D = 2, 300, 64
    b = R.Batch("bf16", H, D, 64, [N, N], [N, N], seed=7, fill=False)
    k, v, q = (bf16(b.rng.standard_normal((2, N, H, D))) for _ in range(3))
    KV.append(b.cache, k.view(2 * N, H, D), v.view(2 * N, H, D), *b.args())
    kd, vd = KV.read(b.cache, b.kv_len, b.block_table, N, layout="NHD")
    assert torch.equal(S.attention(q, kd, vd, causal=True, layout="NHD"), S.attention(q, k, v, causal=True, layout="NHD"))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("inter,rot", [(False, 64), (True, 32)])
def test_a_layer_serves_a_prompt_a_chunk_and_captured_tokens(fmt, inter, rot):
    # the projection's packed rows through norm and rotation into the cache and
    # over it: prompts of odd lengths, a second chunk of one of them, then single
    # tokens from one captured graph; each stage against the plain forms
    from bit_attention_gb300 import qk_rope as Q
    H, Hq, D = 2, 6, 64
    b = R.Batch(fmt, H, D, 16, [45, 130], [45, 130], seed=21, spare=12, fill=False)
    free = sorted(set(range(b.cache.num_pages)) - set(b.table[b.table >= 0]))
    b.table = np.concatenate([b.table, np.full((2, 8), -1)], 1)
    for s, n in ((0, 3), (1, 9)):
        b.table[s, n:n + 4] = [free.pop() for _ in range(4)]
    b.block_table = torch.from_numpy(b.table.astype(np.int32)).cuda()
    table = Q.rope_table(400, rot, scaling="linear", factor=2.0)
    w = [torch.from_numpy(1 + 0.2 * b.rng.standard_normal(D)).bfloat16().cuda() for _ in range(2)]
    rows = bf16(np.zeros((175, Hq + 2 * H, D)))
    pos = torch.zeros(175, dtype=torch.int32, device="cuda")

    def layer(T):
        x = rows[:T]
        qr, kr = Q.forward(x[:, :Hq], x[:, Hq:Hq + H], pos[:T], table, *w, interleaved=inter)
        KV.append(b.cache, kr, x[:, Hq + H:], *b.args())
        return qr, kr, KV.attention(qr, b.cache, *b.args(), return_lse=True)

    def feed(q_lens, kv_lens):
        b.q_lens, b.kv_lens, b.T = q_lens, kv_lens, sum(q_lens)
        b.cu = np.concatenate([[0], np.cumsum(q_lens)])
        b.cu_q.copy_(torch.from_numpy(b.cu.astype(np.int32)))
        b.kv_len.copy_(torch.tensor(kv_lens, dtype=torch.int32))
        p = np.concatenate([np.arange(n - nq, n) for nq, n in zip(q_lens, kv_lens)])
        pos[:b.T].copy_(torch.from_numpy(p.astype(np.int32)))
        rows[:b.T].copy_(bf16(2 * b.rng.standard_normal((b.T, Hq + 2 * H, D))))
        return p

    def check(p, qr, kr, got):
        cos, sin = R.rope_angles(p, rot, scaling="linear", factor=2.0)
        for y, x, wx in ((qr, rows[:b.T, :Hq], w[0]), (kr, rows[:b.T, Hq:Hq + H], w[1])):
            ref = R.rope(R.f64(x), cos, sin, rot, inter, R.f64(wx))
            tol = R.HALF_STEP * np.abs(ref) + 2.0 ** -17 * np.abs(ref).max(-1, keepdims=True)
            assert (np.abs(R.f64(y) - ref) <= tol).all()
        for s in range(2):  # what was stored is the rule's value of what was handed in
            new = slice(b.kv_lens[s] - b.q_lens[s], None)
            for which, part in (("k", kr), ("v", rows[:b.T, Hq + H:])):
                x = R.f64(part[b.cu[s]:b.cu[s + 1]])
                want = x if fmt == "bf16" else R.values(*(torch.from_numpy(t) for t in R.store(x, fmt)), fmt)
                assert np.array_equal(b.dense(which, s)[:, new], want.transpose(1, 0, 2))
        R.check_attention(b, qr, *got)

    for q_lens, kv_lens in (([45, 130], [45, 130]), ([20, 0], [65, 130]), ([1, 3], [66, 133])):
        p = feed(q_lens, kv_lens)
        check(p, *layer(b.T))
    feed([1, 1], [67, 134])
    layer(2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(2)
    for i in range(3):
        p = feed([1, 1], [67 + i, 134 + i])
        graph.replay()
        torch.cuda.synchronize()
        check(p, *out)
    k, v = KV.read(b.cache, b.kv_len, b.block_table, 136)
    assert np.array_equal(R.f64(k[1, :, :136]), b.dense("k", 1)[:, :136])
    assert table.get_status() == S.OK and b.cache.get_status() == S.OK


@pytest.mark.parametrize("fmt", FORMATS)
def test_sequences_that_share_pages(fmt):
    # a common prefix of two pages; every sequence goes on with its own
    b = R.Batch(fmt, 2, 64, 64, [1, 70, 1], [200, 198, 129], seed=22)
    b.table[1:, :2] = b.table[0, :2]
    b.block_table.copy_(torch.from_numpy(b.table.astype(np.int32)))
    q = bf16(b.rng.standard_normal((b.T, 4, 64)))
    R.check_attention(b, q, *KV.attention(q, b.cache, *b.args(), return_lse=True))


@pytest.mark.parametrize("q_of,G", [(lambda s: 1, 2), (lambda s: (s * 7) % 5, 2), (lambda s: 40 if s % 3 == 0 else 0, 1)])
def test_more_sequences_than_one_round_of_the_plan(q_of, G):
    # several of them empty, in the cache or in the batch
    n = 1100
    q_lens = [q_of(s) for s in range(n)]
    kv_lens = [max(q, (s * 13) % 90) if s % 11 else q for s, q in enumerate(q_lens)]
    b = R.Batch("nvfp4", 1, 64, 16, q_lens, kv_lens, seed=23)
    q = bf16(b.rng.standard_normal((b.T, G, 64)))
    R.check_attention(b, q, *KV.attention(q, b.cache, *b.args(), return_lse=True))
    kv = bf16(b.rng.standard_normal((b.T, 2, 64)))
    KV.append(b.cache, kv[:, :1], kv[:, 1:], *b.args())
    for s in range(0, n, 97):
        if q_lens[s]:
            x, sc = (torch.from_numpy(t) for t in R.store(R.f64(kv[b.cu[s]:b.cu[s + 1], :1]), "nvfp4"))
            assert np.array_equal(b.dense("k", s)[:, kv_lens[s] - q_lens[s]:], R.values(x, sc, "nvfp4").transpose(1, 0, 2))
    assert b.cache.get_status() == S.OK


def test_one_long_prompt_among_many_empty_sequences():
    # few rows a sequence on average, more row tiles of one than a round of the plan
    n = 1024
    q_lens, kv_lens = [0] * n, [(s * 5) % 40 for s in range(n)]
    q_lens[700], kv_lens[700] = 5000, 5003
    b = R.Batch("bf16", 1, 64, 64, q_lens, kv_lens, seed=28)
    q = bf16(b.rng.standard_normal((b.T, 2, 64)))
    for window in (None, 300):
        R.check_attention(b, q, *KV.attention(q, b.cache, *b.args(), window=window, return_lse=True), window=window)
    assert b.cache.get_status() == S.OK


def test_calls_side_by_side_on_two_streams():
    # with a workspace each: chunks on one stream, single tokens on the other
    b = R.Batch("e4m3", 2, 128, 64, [300, 77], [900, 2000], seed=24)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    q, q1 = bf16(b.rng.standard_normal((377, 8, 128))), bf16(b.rng.standard_normal((2, 8, 128)))
    ref, ref1 = KV.attention(q, b.cache, *b.args()), KV.attention(q1, b.cache, one, b.kv_len, b.block_table)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = []
    for _ in range(8):
        out.append((KV.attention(q, b.cache, *b.args(), stream=sides[0]),
                    KV.attention(q1, b.cache, one, b.kv_len, b.block_table, stream=sides[1])))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ref) and torch.equal(y, ref1) for x, y in out) and b.cache.get_status() == S.OK


def test_two_graphs_that_share_a_workspace():
    # replayed one after the other, in both orders
    b = R.Batch("bf16", 2, 64, 16, [200, 1], [300, 500], seed=25)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    q, q1 = bf16(b.rng.standard_normal((201, 4, 64))), bf16(b.rng.standard_normal((2, 4, 64)))
    ws = torch.empty(max(KV.attention_workspace_bytes(b.cache, 2, t, 4) for t in (2, 201)), dtype=torch.uint8, device="cuda")
    calls = [lambda: KV.attention(q, b.cache, *b.args(), workspace=ws),
             lambda: KV.attention(q1, b.cache, one, b.kv_len, b.block_table, workspace=ws)]
    refs = [c().clone() for c in calls]
    graphs, outs = [], []
    for c in calls:
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(c())
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for x in outs:
            x.fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, r) for x, r in zip(outs, refs))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_withheld_signal_sets_timeout_and_the_context_survives(fmt, D):
    b = R.Batch(fmt, 2, D, 16, [300, 50], [900, 700], seed=26)
    q = bf16(b.rng.standard_normal((b.T, 4, D)))
    ref = KV.attention(q, b.cache, *b.args(), scale=0.125)
    assert b.cache.get_status() == S.OK
    out = torch.zeros_like(q)
    nbytes = KV.attention_workspace_bytes(b.cache, 2, b.T, 4)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    rows = KV.sage_kv_rows(4 * D, D)
    batch = KV._batch(b.cache, *b.args())
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    rc = KV.sage_kv_attn_stall_test(b.cache.struct, batch, q.data_ptr(), rows, out.data_ptr(), rows, b.T, 4, 20_000_000,
                                    ws.data_ptr(), nbytes, S._stream())
    end.record()
    assert rc == S.OK
    torch.cuda.synchronize()
    assert 15 < start.elapsed_time(end) < 500  # the 20 ms limit, not the default 1.5 s
    assert b.cache.get_status() == S.ETIMEOUT and b.cache.get_status() == S.OK
    assert torch.equal(KV.attention(q, b.cache, *b.args(), scale=0.125), ref) and b.cache.get_status() == S.OK
    # the rows of the last head's entries lie in other CTAs' shares
    assert torch.equal(out[300:, 3], ref[300:, 3])
    few = KV.sage_kv_attn_stall_test(b.cache.struct, batch, q.data_ptr(), rows, out.data_ptr(), rows, 2, 4, 20_000_000,
                                     ws.data_ptr(), nbytes, S._stream())
    assert few == S.EINVAL


def test_offsets_beyond_32_bits():
    # a cache of more than 2^32 bytes of keys: a sequence on its last pages
    H, D, page = 8, 128, 1024
    pages = (1 << 32) // (H * D * page * 2) + 40  # bf16: 2 MiB a page
    c = KV.PagedCache(pages, page, H, D, "bf16")
    for last in (pages - 1, pages - 20):
        table = torch.tensor([[last, 0]], dtype=torch.int32, device="cuda")
        cu, n = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1500], [1500]))
        g = torch.Generator("cuda").manual_seed(last)
        kv = torch.randn((1500, 2 * H, D), generator=g, device="cuda").to(torch.bfloat16)
        KV.append(c, kv[:, :H], kv[:, H:], cu, n, table)
        k, v = KV.read(c, n, table, 1500, layout="NHD")
        assert torch.equal(k[0], kv[:, :H]) and torch.equal(v[0], kv[:, H:])
        q = torch.randn((1500, H, D), generator=g, device="cuda").to(torch.bfloat16)
        o = KV.attention(q, c, cu, n, table)
        small = KV.PagedCache(2, page, H, D, "bf16")
        t2 = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
        KV.append(small, kv[:, :H], kv[:, H:], cu, n, t2)
        assert torch.equal(o, KV.attention(q, small, cu, n, t2))
    assert c.get_status() == S.OK


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens,G", [([5, 1], [2, 40], 2), ([150, 3], [70, 2], 4)])
def test_the_widest_windows_and_tokens_before_the_first_position(fmt, q_lens, kv_lens, G):
    # more new tokens than the cache holds: their windows begin before any int32
    b = R.Batch(fmt, 2, 64, 16, q_lens, kv_lens, seed=29)
    q = bf16(b.rng.standard_normal((b.T, 2 * G, 64)))
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 60, 30):
        for causal in (True, False):
            o, lse = KV.attention(q, b.cache, *b.args(), causal=causal, window=window, return_lse=True)
            R.check_attention(b, q, o, lse, causal=causal, window=window, label=f"{window} {causal}")
    assert b.cache.get_status() == S.OK


def test_more_rows_than_an_int_counts_are_refused():
    # broadcast rows, so that no memory is behind them
    b = R.Batch("bf16", 2, 64, 16, [3], [3], fill=False)
    one = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    for n in (2 ** 31, 2 ** 32 + 3):
        many = one.expand(n, 2, 64)
        for call in (lambda: KV.append(b.cache, many, many, *b.args()), lambda: KV.attention(many, b.cache, *b.args())):
            with pytest.raises(S.SageFp4Error) as e:
                call()
            assert e.value.code == S.EINVAL
    torch.cuda.synchronize()
    assert torch.isnan(b.cache.k_codes).all() and b.cache.get_status() == S.OK


def test_a_status_is_read_on_its_own_stream():
    # while the default stream is busy with something else
    b = R.Batch("bf16", 2, 64, 16, [3], [3])
    side = torch.cuda.Stream()
    b.cache.status[0] = S.EINDEX
    torch.cuda.synchronize()
    torch.cuda._sleep(500_000_000)
    assert b.cache.get_status(side) == S.EINDEX and b.cache.get_status(side) == S.OK
    assert not torch.cuda.current_stream().query()


def test_first_calls_from_many_threads():
    # of a process: what the library notes of a device is noted by one of them
    import subprocess
    import sys
    code = """
import sys, threading
sys.path[:0] = ["tests", "."]
import kv_reference as R, torch
from bit_attention_gb300 import kv_cache as KV, sage_fp4 as S
shapes = [([1, 1], [70, 300]), ([150, 3], [150, 40])]
n = 16
outs = [None] * n
S.load()
torch.zeros(1, device="cuda")
start, bad = threading.Barrier(n), []
def work(i):
    try:
        start.wait()
        b = R.Batch("e4m3", 2, 64, 16, *shapes[i % 2], seed=i % 2)
        q = torch.ones((b.T, 8, 64), dtype=torch.bfloat16, device="cuda")
        outs[i] = KV.attention(q, b.cache, *b.args())
        assert b.cache.get_status() == S.OK
    except BaseException as e:
        bad.append(e)
threads = [threading.Thread(target=work, args=(i,)) for i in range(n)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not bad, bad
assert all(torch.equal(outs[i], outs[i % 2]) for i in range(n))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=__file__.rsplit("/tests/", 1)[0])
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [([2, 1], [300, 90]), ([140, 20], [300, 90]), ([2, 70], [9000, 70])])
def test_scores_of_any_size(fmt, D, q_lens, kv_lens):
    # one-hot keys of several sizes and queries that hit one channel: scores from
    # 2^8 to 2^100 and below 0, where FP32 has no digits left for what is added to
    # one.  A score is one product, rounded three times in FP32: within 2^-22 of
    # itself.  Keys that lie nearer than that to the row's largest (and 100 for
    # what underflows) may share its weight in any way.
    n, H, G = sum(kv_lens), 1, 8
    b = R.Batch(fmt, H, D, 64, q_lens, kv_lens, seed=30, fill=False)
    k = np.zeros((n, H, D))
    k[np.arange(n), 0, np.arange(n) % D] = np.array([4.0, 6.0, 8.0, 7.0, 12.0])[np.arange(n) // D % 5]
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(kv_lens)]).astype(np.int32)).cuda()
    KV.append(b.cache, bf16(k), bf16(b.rng.standard_normal((n, H, D))), cu, b.kv_len, b.block_table)
    t, h = np.indices((b.T, G))
    alone = 0
    for size in (2.0 ** 8, 2.0 ** 17, 2.0 ** 20, 2.0 ** 24, 2.0 ** 31, 2.0 ** 60, 2.0 ** 100):
        q = np.zeros((b.T, G, D))
        q[t, h, b.rng.integers(0, D, t.shape)] = size * b.rng.choice([-1.0, 1.0], t.shape) * b.rng.uniform(0.5, 1.0, t.shape)
        q = bf16(q)
        o, lse = (R.f64(x) for x in KV.attention(q, b.cache, *b.args(), return_lse=True))
        q = R.f64(q)
        for s, (nq, m) in enumerate(zip(q_lens, kv_lens)):
            kd, vd = b.dense("k", s)[0], b.dense("v", s)[0]
            for i in range(nq):
                seen = m - nq + i + 1
                x = q[b.cu[s] + i] @ kd[:seen].T * D ** -0.5
                top = x.max(-1)
                for g in range(G):
                    near = x[g] >= top[g] - 100 - 2.0 ** -20 * abs(top[g])
                    v, got = vd[:seen][near], o[b.cu[s] + i, g]
                    edge = 2.0 ** -6 * np.abs(v).max(0)  # a weight's rounding, a result's
                    alone += near.sum() == 1
                    assert (got >= v.min(0) - edge).all() and (got <= v.max(0) + edge).all(), (size, s, i, g)
                    assert abs(lse[b.cu[s] + i, g] - top[g]) <= 2.0 ** -20 * abs(top[g]) + np.log(near.sum()) + 1e-5, (size, s, i, g)
    assert alone > 0 and b.cache.get_status() == S.OK


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens", [([2, 1], [700, 300]), ([150, 90], [700, 300]), ([1, 40], [5000, 300])])
def test_scores_that_change_from_huge_to_small_and_back(fmt, q_lens, kv_lens):
    # stretches of 150 keys whose scores are all -A, 0, A or 2A for every query of a
    # head: the last kind that a row sees takes it all, equally
    D, H, G, n = 64, 1, 8, sum(kv_lens)
    b = R.Batch(fmt, H, D, 16, q_lens, kv_lens, seed=31, fill=False)
    k = np.zeros((n, H, D))
    order = np.concatenate([np.arange(m) // 150 % 4 for m in kv_lens])
    k[:, 0, 0] = np.array([-4.0, 0.0, 4.0, 8.0])[order]
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(kv_lens)]).astype(np.int32)).cuda()
    KV.append(b.cache, bf16(k), bf16(b.rng.standard_normal((n, H, D))), cu, b.kv_len, b.block_table)
    q = np.zeros((b.T, G, D))
    q[:, :, 0] = 2.0 ** np.array([10, 20, 22, 26, 30, 40, 70, 100])
    for sign in (1.0, -1.0):
        o = R.f64(KV.attention(bf16(sign * q), b.cache, *b.args()))
        for s, (nq, m) in enumerate(zip(q_lens, kv_lens)):
            kd, vd = b.dense("k", s)[0], b.dense("v", s)[0]
            for i in range(nq):
                x = sign * kd[:m - nq + i + 1, 0]
                v = vd[:m - nq + i + 1][x == x.max()]
                # weights alike but for a rounding each (2^-8), and the result's; FP32 sums of up to 2^12 terms
                tol = (2.0 ** -8 * 1.01 + 2.0 ** -12) * (np.abs(v).mean(0) + np.abs(v.mean(0)))
                assert (np.abs(o[b.cu[s] + i] - v.mean(0)) <= tol).all(), (sign, s, i)
    assert b.cache.get_status() == S.OK


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("nq", [1, 100])
def test_lengths_next_to_the_largest_int_are_recorded_and_left_out(fmt, nq):
    # a table that repeats a page holds any number of tokens; ends of tiles would not
    # be ints any more
    b = R.Batch(fmt, 1, 64, 1024, [nq, nq], [1000, 1000], seed=32)
    table = b.block_table[:, :1].expand(2, 1 << 21).contiguous()
    q = bf16(b.rng.standard_normal((b.T, 2, 64)))
    R.check_attention(b, q, *KV.attention(q, b.cache, b.cu_q, b.kv_len, table, return_lse=True))
    assert b.cache.get_status() == S.OK
    b.kv_lens[0] = 0
    for n in (2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 4095):
        lens = b.kv_len.clone()
        lens[0] = n
        o, lse = KV.attention(q, b.cache, b.cu_q, lens, table, return_lse=True)
        assert b.cache.get_status() == S.EINDEX
        assert (o[:nq] == 0).all() and torch.isneginf(lse[:nq]).all()
        R.check_attention(b, q, o, lse)
        k, v = KV.read(b.cache, lens, table, 64)
        assert b.cache.get_status() == S.EINDEX and (k[0] == 0).all() and (v[0] == 0).all() and (k[1] != 0).any()


def test_outputs_laid_over_inputs_are_refused():
    b = R.Batch("bf16", 2, 64, 16, [3, 200], [20, 300])
    q = bf16(b.rng.standard_normal((b.T, 4, 64)))
    wide = torch.zeros((b.T, 8, 64), dtype=torch.bfloat16, device="cuda")
    dense = torch.zeros((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    cu, n, table = b.args()
    keep = q.clone()
    for call in (lambda: KV.attention(q, b.cache, cu, n, table, out=q),
                 lambda: KV.attention(wide[:, ::2], b.cache, cu, n, table, out=wide[:, :4]),
                 lambda: KV.read(b.cache, n, table, 8, out=(dense, dense))):
        with pytest.raises(S.SageFp4Error) as e:
            call()
        assert e.value.code == S.EINVAL
    assert torch.equal(q, keep) and (dense == 0).all() and b.cache.get_status() == S.OK
    wide[:, :4] = q  # side by side in one tensor they are apart
    KV.attention(wide[:, :4], b.cache, cu, n, table, out=wide[:, 4:])
    assert torch.equal(wide[:, 4:], KV.attention(q, b.cache, cu, n, table))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_lens,kv_lens", [([2], [290]), ([140], [290]), ([140], [2900])])
def test_huge_scores_below_zero_before_others_and_channels_of_zeros(fmt, q_lens, kv_lens):
    # nothing of the first half of the keys, whose scores are far below 0, is left in
    # any channel, whatever the first channels hold
    D, n = 64, kv_lens[0]
    b = R.Batch(fmt, 1, D, 16, q_lens, kv_lens, seed=33, fill=False)
    k, v = np.zeros((n, 1, D)), b.rng.standard_normal((n, 1, D))
    k[:n // 2, 0, 0] = -4.0
    v[:, :, :16] = 0.0
    KV.append(b.cache, bf16(k), bf16(v), torch.tensor([0, n], dtype=torch.int32, device="cuda"), b.kv_len, b.block_table)
    q = np.zeros((b.T, 10, D))
    q[:, :, 0] = 2.0 ** np.array([10, 20, 24, 28, 31, 33, 36, 50, 80, 100])
    o = R.f64(KV.attention(bf16(q), b.cache, *b.args()))
    vd = b.dense("v", 0)[0]
    for i in range(b.T):
        seen = vd[n // 2:n - b.T + i + 1]
        # weights alike but for a rounding each (2^-8), and the result's; FP32 sums of up to 2^11 terms
        tol = (2.0 ** -8 * 1.01 + 2.0 ** -13) * (np.abs(seen).mean(0) + np.abs(seen.mean(0)))
        assert (np.abs(o[i] - seen.mean(0)) <= tol).all(), i
    assert b.cache.get_status() == S.OK
