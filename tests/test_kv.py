"""The 4-bit key/value cache: what dsq_kv_append writes (byte for byte), what
dsq_kv_read gives back (bit for bit) and dsq_kv_attend against attention in 64
bits over the same cache.  Refusals run without a GPU.

Tolerance of attend, element by element, from what its header declares.  With
S = scale * sum_i |q_i k_ti| (largest over the tokens), P = sum_t p_t |v_t|:
  scores: fp32 sums of D products, each step off by at most an ulp (2^-23):
    |error| <= (D + 8) 2^-23 S, which moves each p_t, and their sum, by that
    part of themselves, as 2^-20 covers exp2, its argument's last bits and the
    other fp32 steps: 2 ((D + 8) 2^-23 S + 2^-20) P;
  numerators in fp16: 2^-11 of p_t, or 2^-25 of the running maximum's
    numerator where that is more (subnormal): 2^-11 P + T 2^-25 max |v|
    (2^-32, as the header has it, in the tests by kernel and by small numerators);
  the output's rounding: 2^-11 |out| (fp16), 2^-8 |out| (bf16), or 2^-25.
The log-sum-exp: (D + 8) 2^-23 S + 2^-20 + 2^-22 |lse|.
"""
import ctypes

import numpy as np
import pytest

import dense_sparse_quantized_b200 as dsq
from oracle import kv as okv

torch = pytest.importorskip("torch")

EPS = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


# ------------------------------------------------- the definition, on the CPU

def test_held_values_are_fp16_and_within_half_a_step():
    rng = np.random.default_rng(1)
    for spread in (1e-7, 1e-4, 0.02, 1.0, 300.0, 2e4):
        x = (rng.standard_normal((400, 64)) * spread).astype(np.float16).astype(np.float64)
        x[:40] = np.abs(x[:40])
        codes, scale, zero = okv.encode(x)
        v = okv.values(codes, scale, zero)
        assert np.array_equal(v, v.astype(np.float16).astype(np.float64))
        err = np.abs(v - np.clip(x, -okv.CLAMP, okv.CLAMP)).reshape(400, 2, 32)
        assert np.all(err <= scale[..., None] / 2)
        assert np.array_equal(scale.astype(np.float16).view(np.uint16) & 15, np.zeros((400, 2), np.uint16))


def test_held_values_worked_by_hand():
    x = np.zeros((1, 32))
    codes, scale, zero = okv.encode(x)
    assert scale[0, 0] == 2.0 ** -20 and zero[0, 0] == 0 and not codes.any()
    x[0, 3], x[0, 4], x[0, 5] = 15.0, 7.5, 6.5        # step 1: ties go to the even code
    codes, scale, zero = okv.encode(x)
    assert scale[0, 0] == 1.0 and zero[0, 0] == 0 and list(codes[0, 3:6]) == [15, 8, 6]
    x[0, 0] = -1.0                                     # 16 / 15 up to a multiple of 1/64: 69/64
    codes, scale, zero = okv.encode(x)
    assert scale[0, 0] == 69 / 64 and zero[0, 0] == 1 and codes[0, 3] == 15 and codes[0, 0] == 0
    x[0, 9] = np.nan
    assert np.isnan(okv.held(x)).all()
    assert okv.held(np.full((1, 32), np.inf)).max() <= 61184
    top = okv.held(np.concatenate([np.full((1, 16), 7e4), np.full((1, 16), -7e4)], 1))
    assert np.isfinite(top.astype(np.float16)).all()


def test_store_and_load_agree():
    rng = np.random.default_rng(2)
    cache = rng.integers(0, 256, 3 * 2 * 2 * okv.tile_bytes(64), dtype=np.uint8)
    k, v = rng.standard_normal((2, 5, 2, 64)).astype(np.float16)
    slots = np.array([95, 0, 33, -1, 17])
    okv.store(cache, 2, 64, 32, k, v, slots)
    got = okv.load(cache, 2, 64, 32, slots[slots >= 0])
    assert np.array_equal(got[0], okv.held(k)[slots >= 0]) and np.array_equal(got[1], okv.held(v)[slots >= 0])


# ------------------------------------------------------------------ refusals

def _status(fn, *args):
    return getattr(dsq.library(), fn)(*args)


BAD = dsq.DSQ_ERR_INVALID_ARG
UNS = dsq.DSQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("desc,rc", [
    ((0, 0, 128, 64, 4), BAD), ((0, 8, 128, 0, 4), BAD), ((0, 8, 128, 24, 4), BAD), ((0, 8, 128, 64, -1), BAD),
    ((-1, 8, 128, 64, 4), BAD), ((0, 8, 96, 64, 4), UNS), ((0, 8, 0, 64, 4), UNS), ((0, 1, 64, 1 << 16, 1 << 15), UNS), ((0, 1 << 15, 64, 16, 1 << 16), UNS),
    ((0, 8, 128, 64, 4), dsq.DSQ_OK), ((0, 1, 64, 16, 0), dsq.DSQ_OK)])
def test_bytes_refusals(desc, rc):
    size = ctypes.c_size_t(0)
    d = dsq.KVDesc(*desc)
    assert _status("dsq_kv_bytes", ctypes.byref(d), ctypes.byref(size)) == rc
    assert _status("dsq_kv_bytes", None, ctypes.byref(size)) == BAD
    assert _status("dsq_kv_bytes", ctypes.byref(d), None) == BAD
    if rc == dsq.DSQ_OK:
        assert size.value == desc[4] * desc[1] * desc[3] // 16 * okv.tile_bytes(desc[2])
    else:  # every call refuses the shape before it looks at anything else
        assert _status("dsq_kv_append", ctypes.byref(d), None, None, None, 0, None) == rc
        assert _status("dsq_kv_read", ctypes.byref(d), None, None, None, 0, None) == rc
        assert _status("dsq_kv_attend", ctypes.byref(d), None, None, None, None, None) == rc


GOOD_ROWS = dict(k=4096, v=8192, k_token=1024, k_head=128, v_token=1024, v_head=128, dtype=0)


@pytest.mark.parametrize("change", [
    dict(k=None), dict(v=None), dict(k=4104), dict(v=8194), dict(k_token=1028), dict(k_head=4), dict(v_token=1023),
    dict(v_head=-4), dict(dtype=3), dict(dtype=-1)])
def test_append_refusals(change):
    d = dsq.KVDesc(0, 8, 128, 64, 4)
    r = dsq.KVRows(**{**GOOD_ROWS, **change})
    assert _status("dsq_kv_append", ctypes.byref(d), 1 << 20, ctypes.byref(r), 1 << 16, 3, None) == BAD


def test_append_refuses_the_rest():
    d, r = dsq.KVDesc(0, 8, 128, 64, 4), dsq.KVRows(**GOOD_ROWS)
    call = lambda cache, rows, slots, n: _status("dsq_kv_append", ctypes.byref(d), cache, rows, slots, n, None)  # noqa: E731
    assert call(None, ctypes.byref(r), 1 << 16, 3) == BAD
    assert call((1 << 20) + 16, ctypes.byref(r), 1 << 16, 3) == BAD
    assert call(1 << 20, None, 1 << 16, 3) == BAD
    assert call(1 << 20, ctypes.byref(r), None, 3) == BAD
    assert call(1 << 20, ctypes.byref(r), (1 << 16) + 4, 3) == BAD
    assert call(1 << 20, ctypes.byref(r), 1 << 16, -1) == BAD
    assert call(None, None, None, 0) == dsq.DSQ_OK
    r.dtype = dsq.DTYPE_F32
    assert call(1 << 20, ctypes.byref(r), 1 << 16, 3) == UNS
    wide = dsq.KVDesc(0, 70000, 64, 16, 1)
    r.dtype = 0
    assert _status("dsq_kv_append", ctypes.byref(wide), 1 << 20, ctypes.byref(r), 1 << 16, 3, None) == UNS


@pytest.mark.parametrize("change", [
    dict(k=None, v=None), dict(k=4104), dict(k_token=1028), dict(dtype=3), dict(k_token=0), dict(v_head=64),
    dict(k_token=1016), dict(k_token=-1024), dict(k_token=128, k_head=256)])
def test_read_refusals(change):
    """Misaligned rows, and rows that overlap: three tokens of eight heads."""
    d = dsq.KVDesc(0, 8, 128, 64, 4)
    r = dsq.KVRows(**{**GOOD_ROWS, **change})
    assert _status("dsq_kv_read", ctypes.byref(d), 1 << 20, ctypes.byref(r), 1 << 16, 3, None) == BAD


GOOD_Q = dict(q=4096, out=1 << 21, lse=1 << 22, q_token=2048, q_head=128, out_token=2048, out_head=128, q_tokens=6, dtype=0,
              q_heads=16, batch=3, table_pages=2, causal=1, window=0, scale=0.1, page_table=1 << 16, kv_lens=1 << 17,
              q_start=None)


@pytest.mark.parametrize("change,rc", [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(page_table=None), BAD), (dict(kv_lens=None), BAD),
    (dict(q=4104), BAD), (dict(out=4100), BAD), (dict(lse=2), BAD), (dict(q_start=1026), BAD),
    (dict(page_table=(1 << 16) + 2), BAD), (dict(kv_lens=(1 << 17) + 1), BAD),
    (dict(q_token=2044), BAD), (dict(q_head=1), BAD), (dict(out_token=2052), BAD), (dict(out_head=64), BAD),
    (dict(out_token=0), BAD), (dict(out_token=128), BAD), (dict(q_heads=0), BAD), (dict(q_heads=12), BAD), (dict(batch=-1), BAD),
    (dict(q_tokens=-6), BAD), (dict(q_tokens=7), BAD), (dict(table_pages=-1), BAD), (dict(window=-1), BAD),
    (dict(batch=0), BAD), (dict(window=4, causal=0), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(scale=3e38), BAD),
    (dict(dtype=4), BAD), (dict(dtype=2), UNS), (dict(table_pages=1 << 24), UNS), (dict(q_tokens=3 << 28), UNS),
    (dict(q_tokens=3 << 60), UNS)])
def test_attend_refusals(change, rc):
    d = dsq.KVDesc(0, 8, 128, 64, 4)
    size = ctypes.c_size_t(1 << 40)
    a = dsq.KVQueries(**{**GOOD_Q, **change})
    assert _status("dsq_kv_attend", ctypes.byref(d), 1 << 20, ctypes.byref(a), 1 << 24, ctypes.byref(size), None) == rc


def test_attend_workspace_protocol_and_empty_calls():
    d, a = dsq.KVDesc(0, 8, 128, 64, 4), dsq.KVQueries(**GOOD_Q)
    size = ctypes.c_size_t(0)
    call = lambda cache, ws: _status("dsq_kv_attend", ctypes.byref(d), cache, ctypes.byref(a), ws, ctypes.byref(size), None)  # noqa: E731
    assert call(1 << 20, None) == dsq.DSQ_ERR_BUFFER_TOO_SMALL and size.value > 0
    need, size.value = size.value, size.value - 1
    assert call(1 << 20, 1 << 24) == dsq.DSQ_ERR_BUFFER_TOO_SMALL and size.value == need
    assert call(1 << 20, (1 << 24) + 128) == BAD     # misaligned workspace
    assert call((1 << 20) + 64, 1 << 24) == BAD      # misaligned cache
    assert call(None, 1 << 24) == BAD
    assert _status("dsq_kv_attend", ctypes.byref(d), 1 << 20, ctypes.byref(a), 1 << 24, None, None) == BAD
    assert _status("dsq_kv_attend", ctypes.byref(d), 1 << 20, None, 1 << 24, ctypes.byref(size), None) == BAD
    a.batch = a.q_tokens = 0
    assert call(None, 1 << 24) == dsq.DSQ_OK


# --------------------------------------------------------------------- on a GPU

def _rows(rng, n, h, d):
    x = rng.standard_normal((n, h, d)) * np.exp(0.6 * rng.standard_normal((h, d)))
    return torch.from_numpy(x)


def _awkward(x):
    """Groups a quantiser can go wrong in, in the first tokens of x [n, h, d]."""
    n = x.shape[0]
    for i, f in enumerate((lambda g: g * 0, lambda g: g.abs(), lambda g: -g.abs(), lambda g: g * 1e-7, lambda g: g * 3e-5,
                           lambda g: g.clamp(-1, 1) * 65504, lambda g: g * 0 + 1, lambda g: (g * 4).round() / 2,
                           lambda g: torch.where(g == g.max(), float("inf"), g),
                           lambda g: torch.where(g == g.min(), -float("inf"), g),
                           lambda g: torch.where(g == g.max(), float("nan"), g), lambda g: g * 0 - 1e-6)):
        if i < n:
            x[i] = f(x[i])
    return x


def _held(t):
    return okv.held(t.double().cpu().numpy())


CASES = [(1, 1, 64, 16), (3, 2, 64, 32), (33, 8, 128, 16), (40, 3, 128, 48), (29, 1, 256, 128), (513, 2, 128, 64), (700, 12, 64, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,h,d,page", CASES)
def test_append_bytes_and_read_values(n, h, d, page, dtype):
    rng = np.random.default_rng(n + d)
    pages = -(-n // page) + 2
    before = torch.from_numpy(rng.integers(0, 256, dsq.KVCache.bytes_for(h, d, pages, page), dtype=np.uint8))
    kv = dsq.KVCache(h, d, pages, page, data=before.cuda())
    k, v = (_awkward(_rows(rng, n, h, d)).to(dtype) for _ in range(2))
    slots = rng.permutation(pages * page)[:n]
    if n > 20:
        slots[5], slots[17], slots[19] = -1, pages * page, -(1 << 40)
    s = torch.from_numpy(slots).cuda()
    kv.append(k.cuda(), v.cuda(), s)
    want = before.numpy().copy()
    okv.store(want, h, d, page, k.double().numpy(), v.double().numpy(), slots)
    assert np.array_equal(kv.data.cpu().numpy(), want)

    inside = (slots >= 0) & (slots < pages * page)
    exact = okv.load(want, h, d, page, slots[inside])
    for out in (F16, BF16, F32):
        got = kv.read(s, k=torch.full((n, h, d), 7.0, dtype=out, device="cuda"),
                      v=torch.full((n, h, d), 7.0, dtype=out, device="cuda"))
        for g, e in zip(got, exact):
            g = g.cpu()
            assert torch.equal(torch.nan_to_num(g[torch.from_numpy(inside)], 3e4),
                               torch.nan_to_num(torch.from_numpy(e).to(out), 3e4))
            assert (g[torch.from_numpy(~inside)] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["fused", "heads_first", "broadcast", "reversed_tokens"])
def test_append_strides(layout):
    rng = np.random.default_rng(4)
    n, h, d = 21, 4, 128
    if layout == "fused":
        x = _rows(rng, n, 3 * h, d).half().cuda()
        k, v = x[:, h:2 * h], x[:, 2 * h:]
    elif layout == "heads_first":
        k, v = (_rows(rng, h, n, d).half().cuda().transpose(0, 1) for _ in range(2))
    elif layout == "broadcast":
        k, v = _rows(rng, n, 1, d).half().cuda().expand(n, h, d), _rows(rng, 1, h, d).half().cuda().expand(n, h, d)
    else:  # negative strides reach the C call only
        k, v = (_rows(rng, n, h, d).half().cuda() for _ in range(2))
    kv = dsq.KVCache(h, d, 2, 16)
    slots = torch.from_numpy(rng.permutation(32)[:n]).cuda()
    if layout == "reversed_tokens":
        last = (n - 1) * h * d * 2
        r = dsq.KVRows(k.data_ptr() + last, v.data_ptr() + last, -h * d, d, -h * d, d, 0)
        rc = dsq.library().dsq_kv_append(ctypes.byref(kv.desc), kv.data.data_ptr(), ctypes.byref(r), slots.data_ptr(), n,
                                         torch.cuda.current_stream().cuda_stream)
        assert rc == dsq.DSQ_OK
        k, v = k.flip(0), v.flip(0)
    else:
        kv.append(k, v, slots)
    into = torch.zeros(h, n, 2, d, dtype=F32, device="cuda")       # read back into strided views of one tensor
    got = kv.read(slots, k=into[:, :, 0].transpose(0, 1), v=into[:, :, 1].transpose(0, 1))
    assert np.array_equal(got[0].cpu().double().numpy(), _held(k)) and np.array_equal(got[1].cpu().double().numpy(), _held(v))


@pytest.mark.gpu
def test_read_of_keys_alone_and_of_repeated_slots():
    rng = np.random.default_rng(5)
    kv = dsq.KVCache(2, 64, 2, 16)
    k, v = _rows(rng, 9, 2, 64).half().cuda(), _rows(rng, 9, 2, 64).half().cuda()
    kv.append(k, v, torch.arange(9, device="cuda"))
    slots = torch.tensor([8, 3, 3, 0, 8], device="cuda")
    out = torch.zeros(5, 2, 64, dtype=F16, device="cuda")
    for which, x in (("k", k), ("v", v)):
        r = dsq.KVRows(dtype=0, k_token=128, k_head=64, v_token=128, v_head=64)
        setattr(r, which, out.data_ptr())
        assert dsq.library().dsq_kv_read(ctypes.byref(kv.desc), kv.data.data_ptr(), ctypes.byref(r), slots.data_ptr(), 5,
                                         torch.cuda.current_stream().cuda_stream) == dsq.DSQ_OK
        assert np.array_equal(out.cpu().double().numpy(), _held(x[slots]))


def _problem(seed, lens, new, h, share, d, page, dtype, fill=0xFF, extra=2, sizes=None):
    """A cache with the sequences' tokens on shuffled pages; all other bytes are
    `fill` (0xFF: NaN scales).  sizes: what each token's values are multiplied by,
    over and over."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages, cols = sum(need) + extra, max(need + [1])
    data = torch.full((dsq.KVCache.bytes_for(h, d, pages, page),), fill, dtype=torch.uint8, device="cuda")
    kv = dsq.KVCache(h, d, pages, page, data=data)
    order = rng.permutation(pages)
    table = np.full((len(lens), cols), -1, np.int32)
    seqs, at = [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        k, v = _rows(rng, n, h, d), _rows(rng, n, h, d)
        if sizes is not None and n:
            by = torch.tensor(sizes * n)[:n, None, None]
            k, v = k * by, v * by.flip(0)
        k, v = k.to(dtype), v.to(dtype)
        t = np.arange(n)
        if n:
            kv.append(k.cuda(), v.cuda(), torch.from_numpy(table[b, t // page].astype(np.int64) * page + t % page).cuda())
        seqs.append((_held(k), _held(v)))
    rows = sum(new)
    q = torch.from_numpy(rng.standard_normal((rows, h * share, d))).to(dtype)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return kv, seqs, q, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), start


def _check(out, lse, q, seqs, lens, start, dtype, causal=True, window=0, scale=None):
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    for b, (k, v) in enumerate(seqs):
        r0, r1 = int(start[b]), int(start[b + 1])
        if r1 == r0:
            continue
        x = q[r0:r1].double().numpy()
        pos = lens[b] - (r1 - r0) + np.arange(r1 - r0) if causal else None
        want, want_lse, P = okv.attend(x, k, v, scale, pos, window)
        share = x.shape[1] // k.shape[1]
        S = np.zeros(x.shape[:2])
        if lens[b]:
            for h in range(x.shape[1]):
                S[:, h] = abs(scale) * (np.abs(x[:, h]) @ np.abs(k[:, h // share]).T).max(-1)
        ds = (d + 8) * 2.0 ** -23 * S
        tol = (2 * (ds + 2.0 ** -20) + 2.0 ** -11)[..., None] * P + (lens[b] * 2.0 ** -25 * np.abs(v).max(initial=0)
                                                                    + EPS[dtype] * np.abs(want) + 2.0 ** -25)
        err = np.abs(out[r0:r1].double().cpu().numpy() - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        if lse is not None:
            got = lse[r0:r1].double().cpu().numpy()
            empty = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(got), empty), b
            off = np.abs(got[~empty] - want_lse[~empty])
            assert np.all(off <= ds[~empty] + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse[~empty])), (b, off.max())
            assert not out[r0:r1].cpu()[torch.from_numpy(empty)].any()


SHAPES = [  # lens, new rows, kv heads, share, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 17, 0, 255], [1, 1, 1, 1], 2, 1, 128, 16),
    ([333], [1], 32, 1, 128, 64),
    ([100, 1500, 31, 16], [1, 1, 1, 1], 2, 4, 128, 64),
    ([777, 64], [1, 1], 1, 16, 256, 128),
    ([2100], [1], 1, 71, 64, 32),
    ([50, 513, 8], [4, 5, 8], 2, 8, 128, 16),
    ([5, 40], [3, 2], 3, 7, 64, 48),
    ([300], [300], 2, 4, 128, 64),
    ([130, 3, 260, 0], [130, 2, 77, 0], 2, 2, 64, 16),
    ([1000], [129], 1, 1, 256, 32),
    ([4, 10, 129], [9, 10, 129], 1, 3, 128, 16),   # more queries than tokens: the first see nothing
    ([700], [260], 1, 8, 256, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attend_causal(case, dtype):
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case, lens, new, h, share, d, page, dtype)
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), return_lse=True)
    _check(out, lse, q, seqs, lens, start, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [1, 3, 6, 9, 11])
def test_attend_all_tokens(case):
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case + 50, lens, new, h, share, d, page, F16)
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), causal=False, return_lse=True,
                         scale=0.2)
    _check(out, lse, q, seqs, lens, start, F16, causal=False, scale=0.2)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 16, 100, 1000])
@pytest.mark.parametrize("case", [1, 3, 6, 9, 10, 11])
def test_attend_window(case, window):
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case + 100, lens, new, h, share, d, page, BF16)
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), window=window, return_lse=True)
    _check(out, lse, q, seqs, lens, start, BF16, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 6, 200])
def test_attend_uniform_rows_and_strides(new):
    """q_start left out; q a slice of a fused projection, out heads first."""
    lens, h, share, d = [new + 150, new, new + 4], 2, 4, 128
    kv, seqs, q, table, kv_lens, start = _problem(200 + new, lens, [new] * 3, h, share, d, 32, F16)
    fused = torch.zeros(3 * new, 12, d, dtype=F16, device="cuda")
    fused[:, 2:10] = q.cuda()
    out = torch.zeros(8, 3 * new, d, dtype=F16, device="cuda").transpose(0, 1)
    got = kv.attend(fused[:, 2:10], table, kv_lens, out=out)
    assert got is out
    _check(out, None, q, seqs, lens, start, F16)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [3, 6, 8])
def test_attend_large_and_small_scores(case):
    """Queries that pick out one token, and ones that see all tokens alike."""
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case + 300, lens, new, h, share, d, page, F16)
    q[::2] *= 40
    q[1::2] *= 1e-4
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), return_lse=True)
    _check(out, lse, q, seqs, lens, start, F16)


@pytest.mark.gpu
@pytest.mark.parametrize("factor", [1e-12, 1e-6, 1e10])
def test_attend_bf16_queries_outside_fp16(factor):
    """bf16 rows whose values fp16 could not hold, the scale making up for it."""
    for case in (3, 8):
        lens, new, h, share, d, page = SHAPES[case]
        kv, seqs, q, table, kv_lens, start = _problem(case + 350, lens, new, h, share, d, page, BF16)
        q = (q.double() * factor).to(BF16)
        scale = float(d ** -0.5 / factor)
        out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), return_lse=True, scale=scale)
        _check(out, lse, q, seqs, lens, start, BF16, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 4, 90])
def test_attend_rows_behind_the_last_sequence_and_bad_pages(new):
    lens = [new + 30, new + 200]
    kv, seqs, q, table, kv_lens, start = _problem(400 + new, lens, [new, new], 2, 4, 64, 16, F16)
    more = torch.zeros(2 * new + 5, 8, 64, dtype=F16)
    more[:2 * new] = q
    out = torch.full_like(more, 3.0).cuda()
    lse = torch.full(more.shape[:2], 5.0, device="cuda")
    kv.attend(more.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), out=out, lse=lse)
    _check(out, lse, q, seqs, lens, start, F16)
    assert (out[2 * new:] == 3.0).all() and (lse[2 * new:] == 5.0).all()
    # a page outside the cache is not seen: as if its tokens were not there
    table[1, 2] = kv.pages
    table[1, 4] = -7
    t = np.arange(lens[1])
    keep = (t // 16 != 2) & (t // 16 != 4)
    out = kv.attend(q.cuda(), table, kv_lens, causal=False)
    seqs[1] = tuple(x[keep] for x in seqs[1])
    lens[1] = int(keep.sum())
    _check(out, None, q, seqs, lens, start, F16, causal=False)
    # lengths past the table and below zero are clamped
    out, lse = kv.attend(q.cuda(), table[:, :1].contiguous(), torch.tensor([1 << 30, -4], dtype=torch.int32, device="cuda"),
                         causal=False, return_lse=True)
    _check(out, lse, q, [tuple(x[:16] for x in seqs[0]), tuple(x[:0] for x in seqs[1])], [16, 0], start, F16, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 3, 150])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_nan_stays_where_it_is_seen(new, d):
    """A NaN token reaches the queries at and behind it, no other."""
    n = 150
    kv, seqs, q, table, kv_lens, start = _problem(500 + new, [n], [new], 1, 2, d, 64, F16)
    clean = kv.attend(q.cuda(), table, kv_lens)
    at = n - new + new // 2
    for which in (0, 1):
        kv2 = dsq.KVCache(1, d, kv.pages, 64, data=kv.data.clone())
        slot = int(table[0, at // 64]) * 64 + at % 64
        k, v = (torch.from_numpy(x[at:at + 1]).half().cuda() for x in seqs[0])
        (k, v)[which][0, 0, 40] = float("nan")
        kv2.append(k, v, torch.tensor([slot], device="cuda"))
        out, lse = kv2.attend(q.cuda(), table, kv_lens, return_lse=True)
        assert torch.equal(out[:new // 2], clean[:new // 2])
        hit = out[new // 2:]
        assert torch.isnan(hit).any(-1).all()
        if which == 0:
            assert torch.isnan(hit).all() and torch.isnan(lse[new // 2:]).all()
        else:
            assert torch.isnan(hit[..., 32:64]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [3, 6, 8])
def test_attend_workspace_contents_do_not_matter_and_bits_repeat(case):
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case + 600, lens, new, h, share, d, page, F16)
    q, start = q.cuda(), torch.from_numpy(start).cuda()
    work = kv.attend_workspace(q.shape[0], q.shape[1], len(lens))
    first = None
    for fill in (0, 0xFF, 0x7C):
        work.fill_(fill)
        out, lse = kv.attend(q, table, kv_lens, q_start=start, return_lse=True, workspace=work)
        first = first or (out.clone(), lse.clone())
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        for _ in range(4):
            outs.append(kv.attend(q, table, kv_lens, q_start=start, stream=s, out=torch.zeros_like(q),
                                  workspace=kv.attend_workspace(q.shape[0], q.shape[1], len(lens))))
    torch.cuda.synchronize()


def _check_on_gpu(out, lse, q, seqs, lens, start, dtype, window=0):
    """_check's bounds for long causal sequences, the 64-bit attention on the GPU."""
    d = q.shape[-1]
    for b, (k, v) in enumerate(seqs):
        r0, r1 = int(start[b]), int(start[b + 1])
        k, v = (torch.from_numpy(x).cuda() for x in (k, v))
        pos = lens[b] - (r1 - r0) + torch.arange(r1 - r0, device="cuda")[:, None]
        t = torch.arange(lens[b], device="cuda")
        seen = (t <= pos) & ((t > pos - window) if window else (t >= 0))
        share = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            x, kh, vh = q[r0:r1, h].double().cuda(), k[:, h // share], v[:, h // share]
            y = (x @ kh.T * d ** -0.5).masked_fill(~seen, -torch.inf)
            total = torch.logsumexp(y, -1)
            p = torch.where(seen, torch.exp(y - total[:, None]), 0.0)
            want, P = p @ vh, p @ vh.abs()
            ds = (d + 8) * 2.0 ** -23 * (x.abs() @ kh.abs().T * d ** -0.5).amax(-1)
            tol = (2 * (ds + 2.0 ** -20) + 2.0 ** -11)[:, None] * P + (lens[b] * 2.0 ** -25 * vh.abs().max()
                                                                      + EPS[dtype] * want.abs() + 2.0 ** -25)
            assert bool(((out[r0:r1, h].double() - want).abs() <= tol).all()), (b, h)
            off = (lse[r0:r1, h].double() - total).abs()
            assert bool((off <= ds + 2.0 ** -20 + 2.0 ** -22 * total.abs()).all()), (b, h, float(off.max()))


LONG = [  # lens, new rows, kv heads, share, dim, page, window
    ([3000], [1500], 4, 8, 128, 64, 0),                # many jobs a CTA, joined across CTAs
    ([1400, 900, 33, 2300], [700, 900, 20, 130], 6, 3, 64, 16, 0),
    ([2500, 2049], [400, 513], 2, 4, 256, 32, 0),
    ([6000, 130, 4000], [37, 21, 64], 2, 2, 128, 48, 0),   # jobs of one row tile, shared by units
    ([5000], [1100], 3, 1, 128, 128, 300),
    ([4000, 5000], [1, 1], 5, 8, 128, 64, 0),
    ([9000, 17, 3000], [2, 1, 2], 3, 8, 64, 32, 0),
    ([7000], [1], 1, 16, 256, 16, 0),
    ([1300] * 40, [1] * 40, 8, 4, 128, 64, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(LONG)))
def test_attend_long_and_joined(case):
    lens, new, h, share, d, page, window = LONG[case]
    dtype = (F16, BF16)[case % 2]
    kv, seqs, q, table, kv_lens, start = _problem(700 + case, lens, new, h, share, d, page, dtype)
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), return_lse=True, window=window)
    _check_on_gpu(out, lse, q, seqs, lens, start, dtype, window)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 7, 300])
def test_attend_window_of_any_size(new):
    """A window past every position, the largest number among them, is none."""
    kv, seqs, q, table, kv_lens, start = _problem(860 + new, [new // 2, 400], [new, new], 1, 3, 64, 16, F16)
    q = q.cuda()
    want = kv.attend(q, table, kv_lens)
    for window in (401, 1 << 30, (1 << 31) - 1):
        assert torch.equal(kv.attend(q, table, kv_lens, window=window), want)


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[0.004], [300.0], [1.0] * 64 + [0.003] * 40 + [50.0] * 7 + [2e-6], [1.0, 1.0, 9.0], [1e4]])
@pytest.mark.parametrize("case", [3, 4, 5, 6, 8])
def test_attend_small_and_large_values(case, sizes):
    """Scales from the smallest to the largest, in one run of tokens and side by side."""
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case + 900, lens, new, h, share, d, page, F16, sizes=sizes)
    scale = float(d ** -0.5 / max(sizes))
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), scale=scale, return_lse=True)
    _check(out, lse, q, seqs, lens, start, F16, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("case", [3, 8])
def test_attend_scales_of_zero_and_below(case, scale):
    lens, new, h, share, d, page = SHAPES[case]
    kv, seqs, q, table, kv_lens, start = _problem(case + 800, lens, new, h, share, d, page, F16)
    out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), scale=scale, return_lse=True)
    _check(out, lse, q, seqs, lens, start, F16, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [4, 100])
def test_a_query_of_nan_spoils_its_own_row_alone(new):
    kv, seqs, q, table, kv_lens, start = _problem(850 + new, [600], [new], 2, 2, 128, 64, BF16)
    clean = kv.attend(q.cuda(), table, kv_lens)
    q[new // 2, 1, 5] = float("nan")
    out = kv.attend(q.cuda(), table, kv_lens)
    assert torch.isnan(out[new // 2, 1]).all()
    out[new // 2, 1] = clean[new // 2, 1]
    assert torch.equal(out, clean)


@pytest.mark.gpu
def test_new_tensors_of_a_side_stream_are_made_on_it():
    """Calls on another stream than the current one, which is kept busy: what they
    return is zeroed and filled in their own stream's order."""
    kv, seqs, q, table, kv_lens, start = _problem(870, [300, 40], [1, 1], 2, 4, 64, 16, F16)
    q, more = q.cuda(), torch.zeros(7, 8, 64, dtype=F16, device="cuda")
    more[:2] = q
    qs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    slots = torch.tensor([int(table[0, 0]) * 16, -1], device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = kv.attend(q, table, kv_lens)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            busy = busy @ busy * 1e-3
        out, lse = kv.attend(more, table, kv_lens, q_start=qs, return_lse=True, stream=stream)
        k, v = kv.read(slots, stream=stream)
        side.synchronize()
        with torch.cuda.stream(side):
            assert torch.equal(out[:2], want) and not out[2:].any() and not lse[2:].any()
            assert not k[1].any() and np.array_equal(k[0].double().cpu().numpy(), seqs[0][0][0])
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_far_pages_of_a_large_cache():
    """Byte offsets past 32 bits: a 4.9 GB cache whose first and last pages are used."""
    h, d, page = 8, 128, 64
    pages = 66000
    kv = dsq.KVCache(h, d, pages, page, data=torch.empty(dsq.KVCache.bytes_for(h, d, pages, page), dtype=torch.uint8, device="cuda"))
    assert kv.data.numel() > 1 << 32
    rng = np.random.default_rng(9)
    k, v = _rows(rng, 100, h, d).half(), _rows(rng, 100, h, d).half()
    slots = torch.cat([torch.arange(64) + (pages - 1) * page, torch.arange(36)]).cuda()
    kv.append(k.cuda(), v.cuda(), slots)
    got = kv.read(slots, dtype=F32)
    assert np.array_equal(got[0].cpu().double().numpy(), _held(k)) and np.array_equal(got[1].cpu().double().numpy(), _held(v))
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    for new in (1, 60):
        q = torch.from_numpy(rng.standard_normal((new, 16, d))).half()
        out, lse = kv.attend(q.cuda(), table, torch.tensor([100], dtype=torch.int32, device="cuda"), return_lse=True)
        _check(out, lse, q, [(_held(k), _held(v))], [100], [0, new], F16)


@pytest.mark.gpu
def test_captured_calls_follow_their_buffers():
    """append and attend captured once and replayed over changing rows, slots,
    lengths and pages; two graphs with a workspace each, replayed in turn."""
    rng = np.random.default_rng(11)
    h, share, d, page, batch = 2, 4, 128, 16, 3
    kv = dsq.KVCache(h, d, 40, page)
    table = torch.from_numpy(rng.permutation(40)[:36].reshape(batch, 12).astype(np.int32)).cuda()
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(batch, h, d, dtype=F16, device="cuda") for _ in range(2))
    q = torch.zeros(batch, h * share, d, dtype=F16, device="cuda")
    slots = torch.zeros(batch, dtype=torch.int64, device="cuda")
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for _ in range(2):
        work, out = kv.attend_workspace(batch, h * share, batch), torch.zeros_like(q)
        with torch.cuda.stream(side):
            kv.append(k, v, slots)
            kv.attend(q, table, lens, out=out, workspace=work)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kv.append(k, v, slots)
            kv.attend(q, table, lens, out=out, workspace=work)
        graphs.append((g, work))
        outs.append(out)
    host, tab = np.array([0, 30, 170]), table.cpu().numpy()
    held = [[np.zeros((n, h, d)), np.zeros((n, h, d))] for n in host]
    kv.data.zero_()     # zero words: scale 0, values 0
    for step in range(6):
        new = [_rows(rng, batch, h, d).half() for _ in range(2)]
        x = torch.from_numpy(rng.standard_normal(q.shape)).half()
        slots.copy_(torch.from_numpy(np.array([tab[b, host[b] // page] * page + host[b] % page for b in range(batch)])))
        for b in range(batch):
            held[b] = [np.concatenate([held[b][i], _held(new[i][b:b + 1])]) for i in range(2)]
        host = host + 1
        lens.copy_(torch.from_numpy(host.astype(np.int32)))
        k.copy_(new[0])
        v.copy_(new[1])
        q.copy_(x)
        graphs[step % 2][0].replay()
        _check(outs[step % 2], None, x, held, host, range(batch + 1), F16)


@pytest.mark.gpu
def test_decode_steps_with_quantized_projections(orc):
    """The operators as a layer uses them: q, k and v from quantised matrices
    (Handle.gemv), appended and attended over, and the result through another
    quantised matrix; every step against the oracles on the values it was given."""
    import synth
    h, heads, d, hidden, batch = 2, 4, 64, 256, 2
    mats = {n: synth.make_problem(rows, cols, 3, "affine", 0.01, "uniform", s, batch)
            for n, rows, cols, s in (("q", heads * d, hidden, 1), ("k", h * d, hidden, 2), ("v", h * d, hidden, 3),
                                     ("o", hidden, heads * d, 4))}
    handles = {n: dsq.Handle(dsq.pack_problem(p)) for n, p in mats.items()}
    kv = dsq.KVCache(h, d, 8, 16)
    table = torch.tensor([[5, 0, 2], [7, 1, 3]], dtype=torch.int32, device="cuda")
    held = [[np.zeros((0, h, d)), np.zeros((0, h, d))] for _ in range(batch)]
    rng = np.random.default_rng(20)
    for step in range(20):
        x = torch.from_numpy(rng.standard_normal((batch, hidden)) * 3).half().cuda()
        q, k, v = (handles[n].gemv(x).view(batch, -1, d) for n in "qkv")
        slots = table[:, step // 16].long() * 16 + step % 16
        kv.append(k, v, slots)
        y, lse = kv.attend(q, table, torch.full((batch,), step + 1, dtype=torch.int32, device="cuda"), return_lse=True)
        out = handles["o"].gemv(y.reshape(batch, heads * d))
        for b in range(batch):
            held[b] = [np.concatenate([held[b][i], _held((k, v)[i][b:b + 1])]) for i in range(2)]
        _check(y, lse, q.cpu(), held, [step + 1] * batch, range(batch + 1), F16)
        mats["o"].x = y.reshape(batch, heads * d).cpu().view(torch.int16).numpy().view(np.uint16)
        want, bound = orc.gemv(mats["o"])
        assert np.all(np.abs(out.cpu().double().numpy() - want) <= 1e-3 * bound)
    for p in handles.values():
        p.close()


@pytest.mark.gpu
def test_binding_refusals():
    kv = dsq.KVCache(2, 64, 2, 16)
    k = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    s = torch.arange(3, device="cuda")
    t, n = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    for call in (lambda: kv.append(k, k.float(), s), lambda: kv.append(k, k, s.int()), lambda: kv.append(k[:2], k, s),
                 lambda: kv.append(k.cpu(), k, s), lambda: kv.append(k.transpose(1, 2), k, s),
                 lambda: kv.read(s, k=k, v=k.float()), lambda: kv.read(s[::2]),
                 lambda: kv.attend(k, t, n.long()), lambda: kv.attend(k, t[:2], n), lambda: kv.attend(k[0], t, n),
                 lambda: kv.attend(k, t, n, out=k.float()), lambda: kv.attend(k, t, n, lse=n.float()),
                 lambda: kv.attend(k, t, n, q_start=n), lambda: kv.attend(k.double(), t, n),
                 lambda: dsq.KVCache(2, 64, 2, 16, data=torch.zeros(5, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call, rc in ((lambda: kv.append(k.float(), k.float(), s), UNS), (lambda: kv.attend(k.float(), t, n), UNS),
                     (lambda: kv.attend(k[:, :1].contiguous(), t, n), BAD), (lambda: kv.attend(k, t[:2], n[:2]), BAD),
                     (lambda: kv.attend(k, t, n, window=3, causal=False), BAD),
                     (lambda: kv.attend(k, t, n, scale=float("inf")), BAD),
                     (lambda: kv.attend(k, t, n, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")),
                      dsq.DSQ_ERR_BUFFER_TOO_SMALL)):
        with pytest.raises(dsq.DSQError) as e:
            call()
        assert e.value.status == rc


@pytest.mark.gpu
def test_a_failed_call_is_its_own_failure():
    """An unknown device fails that call, not the library's next one."""
    kv = dsq.KVCache(2, 64, 2, 16)
    k = torch.zeros(3, 2, 64, dtype=F16, device="cuda")
    s = torch.arange(3, device="cuda")
    t, n = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    work = kv.attend_workspace(3, 2, 3)
    w = torch.arange(16 * 64, dtype=F32, device="cuda").view(16, 64)
    for call in (lambda: kv.append(k, k, s), lambda: kv.read(s), lambda: kv.attend(k, t, n, workspace=work)):
        kv.desc.device = 99
        with pytest.raises(dsq.DSQError) as e:
            call()
        assert e.value.status == dsq.DSQ_ERR_CUDA
        kv.desc.device = 0
        dsq.decompose(w, 4, "affine", 8)
        call()


def test_check_refusals():
    for desc, rc in (((0, 0, 128, 64, 4), BAD), ((-1, 8, 128, 64, 4), BAD), ((0, 8, 96, 64, 4), UNS)):
        d = dsq.KVDesc(*desc)
        assert _status("dsq_kv_check", ctypes.byref(d)) == rc
        assert _status("dsq_kv_selftest_wait_timeout", ctypes.byref(d), None) == rc
    assert _status("dsq_kv_check", None) == BAD and _status("dsq_kv_selftest_wait_timeout", None, None) == BAD


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported_once():
    """The attention kernels' bounded wait gives up and returns; check() reports it
    once and clears it, on every cache of the device, and the next call works."""
    kv, seqs, q, table, kv_lens, start = _problem(940, [700], [260], 1, 8, 64, 16, F16)
    other = dsq.KVCache(1, 128, 1, 16)
    kv.attend(q.cuda(), table, kv_lens)
    kv.check()
    kv.selftest_wait_timeout()
    with pytest.raises(dsq.DSQError) as e:
        other.check()
    assert e.value.status == dsq.DSQ_ERR_DEVICE
    kv.check()
    side = torch.cuda.Stream()
    kv.selftest_wait_timeout(stream=side)
    out, lse = kv.attend(q.cuda(), table, kv_lens, return_lse=True)
    with pytest.raises(dsq.DSQError):
        kv.check()
    _check(out, lse, q, seqs, [700], start, F16)
    kv.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d,new,share,n", [(64, 1, 1, 333), (128, 1, 8, 333), (256, 1, 2, 500), (128, 5, 4, 333), (64, 5, 5, 40),
                                           (64, 300, 4, 300), (128, 300, 4, 301), (256, 400, 2, 400), (128, 900, 8, 3000)])
def test_attend_tokens_far_below_the_largest(d, new, share, n, dtype):
    """Every 16th token attracts the row and has the value 0; the others, at 2^-25.3
    of it, are the whole output.  Numerators in fp16 are within 2^-11 of
    themselves or 2^-32 of the largest."""
    h, page = 2, 64
    q0 = torch.tensor(25.3 * np.log(2) / 15 * 8).to(dtype)
    attracts = (torch.arange(n) % 16 == 0)[:, None, None]
    k, v = torch.zeros(n, h, d), torch.where(attracts, 0.0, 30720.0).expand(n, h, d)
    k[..., 0] = torch.where(attracts[..., 0], 15.0, 0.0)
    pages = -(-n // page)
    kv = dsq.KVCache(h, d, pages, page)
    kv.append(k.half().cuda(), v.half().contiguous().cuda(), torch.arange(n, device="cuda"))
    q = torch.zeros(new, h * share, d, dtype=dtype)
    q[..., 0] = q0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out, lse = kv.attend(q.cuda(), table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=0.125, return_lse=True)
    pos = n - new + np.arange(new)
    few = n if new == 1 else 64  # rows are alike: some of them
    rows = np.unique(np.linspace(0, new - 1, few).astype(int))
    want, want_lse, P = okv.attend(q[rows].double().numpy(), k.double().numpy(), v.double().numpy(), 0.125, pos[rows])
    ds = (d + 8) * 2.0 ** -23 * 0.125 * float(q0) * 15
    each = (pos[rows] + 1) / (pos[rows] // 16 + 1)  # tokens seen to one that attracts: their errors' sum over the numerators'
    tol = (2 * (ds + 2.0 ** -20) + 2.0 ** -11) * P + (each * 2.0 ** -32 * 30720)[:, None, None] + EPS[dtype] * np.abs(want) + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy()[rows] - want)
    assert np.all(err <= tol), (float((err / tol).max()), float((err / np.maximum(np.abs(want), 1e-30)).max()))
    off = np.abs(lse.double().cpu().numpy()[rows] - want_lse)
    assert np.all(off <= ds + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse))


@pytest.mark.parametrize("change,rc", [
    (dict(batch=1 << 30), UNS), (dict(batch=1 << 26), UNS), (dict(batch=(1 << 31) - 1, q_heads=8), UNS),
    (dict(batch=(1 << 26) - 1, out=None), BAD)])   # the last is refused for its outputs alone
def test_attend_refuses_more_jobs_than_it_can_number(change, rc):
    """Sequences times kv heads from 2^29 on: the choice of the units' size had no end."""
    d = dsq.KVDesc(0, 8, 128, 64, 4)
    size = ctypes.c_size_t(1 << 40)
    a = dsq.KVQueries(**{**GOOD_Q, "q_start": 1 << 18, **change})
    assert _status("dsq_kv_attend", ctypes.byref(d), 1 << 20, ctypes.byref(a), 1 << 24, ctypes.byref(size), None) == rc


@pytest.mark.gpu
@pytest.mark.parametrize("batch,new,n,window", [
    (6, 40, 200, 0), (6, 300, 400, 0),
    (2896, 8, 23168, 1)])   # 1448 sequences of 23168 rows: 3e9 units of work, more than 31 bits count
def test_attend_row_numbers_out_of_order_touch_nothing_else(batch, new, n, window):
    """q_start 0, N, 0, N, ...: every other sequence has all rows.  What lies around
    the outputs stays as it is, and the next call is right."""
    d, page, rows = 64, 64, batch * new
    rng = np.random.default_rng(batch)
    pages = -(-n // page)
    kv = dsq.KVCache(1, d, pages, page)
    k, v = _rows(rng, n, 1, d).half().cuda(), _rows(rng, n, 1, d).half().cuda()
    kv.append(k, v, torch.arange(n, device="cuda"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(batch, pages).contiguous()
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, rows] * (batch // 2) + [0], dtype=torch.int32, device="cuda")
    q = torch.from_numpy(rng.standard_normal((rows, 1, d))).half().cuda()
    around, lse = torch.full((rows + 2048, 1, d), 3.0, dtype=F16, device="cuda"), torch.full((rows + 2048, 1), 5.0, device="cuda")
    work = torch.full((kv.attend_workspace(rows, 1, batch).numel() + 8192,), 0xAB, dtype=torch.uint8, device="cuda")
    kv.attend(q, table, lens, q_start=start, window=window, out=around[1024:-1024], lse=lse[1024:-1024], workspace=work[:-8192])
    for t, fill in ((around, 3.0), (lse, 5.0)):
        assert (t[:1024] == fill).all() and (t[-1024:] == fill).all()
    assert (work[-8192:] == 0xAB).all()
    few = min(rows, 300)
    out, lse = kv.attend(q[:few], table[:1], lens[:1], window=window, return_lse=True)
    _check(out, lse, q[:few].cpu(), [(_held(k), _held(v))], [n], [0, few], F16, window=window)


@pytest.mark.parametrize("shape", [((1 << 32) + 1, 64, 4, 16), (1, (1 << 32) + 64, 4, 16), (1, 64, 1 << 32, 16),
                                   (1, 64, 4, (1 << 32) + 16), (1, 64, -(1 << 33), 16)])
def test_binding_refuses_sizes_past_32_bits(shape):
    """The bytes of the sizes' low 32 bits were returned."""
    with pytest.raises(ValueError):
        dsq.KVCache.bytes_for(*shape)
    with pytest.raises(ValueError):
        dsq.KVCache(*shape)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 300])
def test_binding_takes_windows_past_32_bits_as_none(new):
    kv, seqs, q, table, kv_lens, start = _problem(960 + new, [600], [new], 1, 3, 64, 16, F16)
    q = q.cuda()
    want = kv.attend(q, table, kv_lens)
    for window in (1 << 31, (1 << 32) + 1, 1 << 32, (1 << 64) + 5):
        assert torch.equal(kv.attend(q, table, kv_lens, window=window), want)
    for window in (-1, -(1 << 32), 3 - (1 << 32)):
        with pytest.raises(dsq.DSQError) as e:
            kv.attend(q, table, kv_lens, window=window)
        assert e.value.status == BAD
    for sizes in ((q.shape[0], 3, 1 << 32), (q.shape[0], (1 << 32) + 3, 1), (1 << 64, 3, 1)):
        with pytest.raises(ValueError):
            kv.attend_workspace(*sizes)


# ------------------------------------------------- each kernel by its own shapes
#
# Which kernel a shape takes follows from estimates of times; the tests below
# state the one that they are for, so that no change of those moves them.

def test_kernel_query_refuses_what_attend_refuses():
    d = dsq.KVDesc(0, 8, 128, 64, 4)
    ask = lambda d, a: _status("dsq_kv_attend_kernel", d and ctypes.byref(d), a and ctypes.byref(a))  # noqa: E731
    assert ask(d, dsq.KVQueries(**GOOD_Q)) in (0, 1)
    for change, rc in ((dict(q_heads=12), BAD), (dict(batch=-1), BAD), (dict(q_tokens=7), BAD), (dict(dtype=2), UNS),
                       (dict(window=4, causal=0), BAD), (dict(table_pages=1 << 24), UNS), (dict(q_tokens=3 << 28), UNS)):
        assert ask(d, dsq.KVQueries(**{**GOOD_Q, **change})) == rc
    assert ask(None, dsq.KVQueries(**GOOD_Q)) == BAD and ask(d, None) == BAD
    assert ask(dsq.KVDesc(0, 8, 96, 64, 4), dsq.KVQueries(**GOOD_Q)) == UNS


def _takes(kv, q, table, ragged=True, **how):
    return kv.attend_kernel(q.shape[0], q.shape[1], table.shape[0], table.shape[1], ragged, **how)


def _check_each(out, lse, q, seqs, lens, start, dtype, causal=True, window=0, scale=None, keep=None):
    """Against attention in 64 bits, worked out on the GPU; the bounds of this file
    with the numerators' 2^-32.  keep: by sequence, the tokens that are there."""
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    for b, (k, v) in enumerate(seqs):
        r0, r1, n = int(start[b]), int(start[b + 1]), int(lens[b])
        if r1 == r0:
            continue
        if n == 0:
            assert not out[r0:r1].any() and (lse is None or torch.isneginf(lse[r0:r1]).all())
            continue
        k, v = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (k, v))
        t = torch.arange(n, device="cuda")
        pos = n - (r1 - r0) + torch.arange(r1 - r0, device="cuda")[:, None]
        seen = (t <= pos) if causal else (t >= 0).expand(r1 - r0, n)
        if window:
            seen = seen & (t > pos - window)
        if keep is not None and keep[b] is not None:
            seen = seen & torch.from_numpy(keep[b]).cuda()
        none = ~seen.any(-1)
        share = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            x, kh, vh = q[r0:r1, h].double().cuda(), k[:, h // share], v[:, h // share]
            y = (x @ kh.T * scale).masked_fill(~seen, -torch.inf)
            total = torch.logsumexp(y, -1)
            p = torch.where(seen, torch.exp(y - total[:, None]), 0.0)
            want, P = p @ vh, p @ vh.abs()
            ds = (d + 8) * 2.0 ** -23 * (x.abs() @ kh.abs().T * abs(scale)).amax(-1)
            tol = (2 * (ds + 2.0 ** -20) + 2.0 ** -11)[:, None] * P + (n * 2.0 ** -32 * vh.abs().max()
                                                                      + EPS[dtype] * want.abs() + 2.0 ** -25)
            err = (out[r0:r1, h].double() - want).abs()
            assert bool((err <= tol).all()), (b, h, float((err / tol).max()))
            assert not out[r0:r1, h][none].any()
            if lse is not None:
                got = lse[r0:r1, h].double()
                assert torch.equal(torch.isneginf(got), none), (b, h)
                off = (got - total)[~none].abs()
                assert bool((off <= (ds + 2.0 ** -20 + 2.0 ** -22 * total.abs())[~none]).all()), (b, h, float(off.max()))


MANY = {  # lens, new rows, kv heads, share, page; for kv_prompt.cu at every head_dim
    "short": ([500, 130, 0, 77, 340], [500, 130, 0, 90, 340], 2, 8, 16),      # a job a CTA; rows that see nothing
    "dealt": ([1900, 700, 0, 1300], [1000, 300, 0, 1300], 3, 4, 64),          # dealt out, joined
    "nine": ([150 * i for i in range(9)], [130 * i for i in range(9)], 2, 4, 32),   # eight sequences and more
    "forty": ([37 * i % 900 for i in range(40)], [min(37 * i % 900, 53 * i % 400) for i in range(40)], 2, 8, 16),
    "halves": ([600, 500, 129, 590, 124, 60, 431, 600], [100, 120, 128, 1, 77, 60, 100, 100], 16, 1, 16),  # up to 128 rows a job
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("name", MANY)
def test_many_rows_causal_all_tokens_and_windows(name, d, dtype):
    lens, new, h, share, page = MANY[name]
    kv, seqs, q, table, kv_lens, start = _problem(1000 + d, lens, new, h, share, d, page, dtype)
    x, qs = q.cuda(), torch.from_numpy(start).cuda()
    for how in (dict(), dict(causal=False), dict(window=1), dict(window=100), dict(window=450)):
        assert _takes(kv, q, table, **how) == "many_rows"
        out, lse = kv.attend(x, table, kv_lens, q_start=qs, return_lse=True, **how)
        _check_each(out, lse, q, seqs, lens, start, dtype, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("name", ["short", "dealt", "halves"])
def test_many_rows_scales_and_values(name, d):
    """Scales of zero and below, tokens of very different sizes, rows that pick out
    one token, bf16 rows that fp16 could not hold."""
    lens, new, h, share, page = MANY[name]
    sizes = [1.0] * 64 + [0.003] * 40 + [50.0] * 7 + [2e-6]
    kv, seqs, q, table, kv_lens, start = _problem(1100 + d, lens, new, h, share, d, page, F16, sizes=sizes)
    qs = torch.from_numpy(start).cuda()
    assert _takes(kv, q, table) == "many_rows"
    for scale in (0.0, -0.3, 0.01):
        out, lse = kv.attend(q.cuda(), table, kv_lens, q_start=qs, scale=scale, return_lse=True)
        _check_each(out, lse, q, seqs, lens, start, F16, scale=scale)
    kv, seqs, q, table, kv_lens, start = _problem(1110 + d, lens, new, h, share, d, page, F16)
    x = q.clone()
    x[::2] *= 40
    x[1::2] *= 1e-4
    out, lse = kv.attend(x.cuda(), table, kv_lens, q_start=qs, return_lse=True)
    _check_each(out, lse, x, seqs, lens, start, F16)
    for factor in (1e-12, 1e10):
        x, scale = (q.double() * factor).to(BF16), float(d ** -0.5 / factor)
        out, lse = kv.attend(x.cuda(), table, kv_lens, q_start=qs, scale=scale, return_lse=True)
        _check_each(out, lse, x, seqs, lens, start, BF16, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("name", ["short", "dealt", "halves"])
def test_many_rows_pages_that_are_not_there(name, d):
    """Page numbers outside the cache, in the middle of sequences; rows behind the last one."""
    lens, new, h, share, page = MANY[name]
    kv, seqs, q, table, kv_lens, start = _problem(1200 + d, lens, new, h, share, d, page, F16)
    keep = [None] * len(lens)
    for b, cols, bad in ((0, (0, 3, 7), kv.pages), (1, (2,), -5), (3, (0, 1), 1 << 30)):
        keep[b] = np.ones(lens[b], bool)
        for c in cols:
            table[b, c] = bad
            keep[b][c * page:(c + 1) * page] = False
    more = torch.zeros(q.shape[0] + 5, *q.shape[1:], dtype=F16)
    more[:-5] = q
    for how in (dict(), dict(causal=False), dict(window=60)):
        assert _takes(kv, more, table, **how) == "many_rows"
        out, lse = torch.full_like(more, 3.0).cuda(), torch.full(more.shape[:2], 5.0, device="cuda")
        kv.attend(more.cuda(), table, kv_lens, q_start=torch.from_numpy(start).cuda(), out=out, lse=lse, **how)
        _check_each(out, lse, q, seqs, lens, start, F16, keep=keep, **how)
        assert (out[-5:] == 3.0).all() and (lse[-5:] == 5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("n,new,h,share", [(900, 700, 4, 8), (400, 400, 2, 8), (400, 100, 64, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_nan_stays_where_it_is_seen(d, n, new, h, share, window):
    """A NaN key or value reaches the rows that see its token and no other, bit for bit."""
    kv, seqs, q, table, kv_lens, start = _problem(1300 + d + n, [n], [new], h, share, d, 64, F16)
    q = q.cuda()
    assert _takes(kv, q, table, ragged=False, window=window) == "many_rows"
    clean, clean_lse = kv.attend(q, table, kv_lens, window=window, return_lse=True)
    pos = n - new + torch.arange(new, device="cuda")
    for at in (n - new + new // 2, n - new // 3 - 16):
        seen = (pos >= at) & ((pos < at + window) if window else (pos >= 0))
        for which in (0, 1):
            kv2 = dsq.KVCache(h, d, kv.pages, 64, data=kv.data.clone())
            k, v = (torch.from_numpy(x[at:at + 1]).half().cuda() for x in seqs[0])
            (k, v)[which][0, :, 40] = float("nan")
            kv2.append(k, v, torch.tensor([int(table[0, at // 64]) * 64 + at % 64], device="cuda"))
            out, lse = kv2.attend(q, table, kv_lens, window=window, return_lse=True)
            assert torch.equal(out[~seen], clean[~seen]) and torch.equal(lse[~seen], clean_lse[~seen])
            assert torch.isnan(out[seen][..., 32:64]).all()
            if which == 0:
                assert torch.isnan(out[seen]).all() and torch.isnan(lse[seen]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_a_query_of_nan_spoils_its_own_row_alone(d):
    for dtype in (F16, BF16):
        kv, seqs, q, table, kv_lens, start = _problem(1400 + d, [900], [500], 4, 8, d, 64, dtype)
        assert _takes(kv, q, table, ragged=False) == "many_rows"
        clean = kv.attend(q.cuda(), table, kv_lens)
        q[250, 1, 5] = float("nan")
        out = kv.attend(q.cuda(), table, kv_lens)
        assert torch.isnan(out[250, 1]).all()
        out[250, 1] = clean[250, 1]
        assert torch.equal(out, clean)


FEW = {  # for kv_split.cu: a job a CTA; dealt out, joined; sixteen rows at once
    "short": ([333, 17, 0, 140], [1, 1, 1, 1], 4, 4, 64),
    "dealt": ([5000, 31, 9000], [1, 1, 1], 2, 8, 64),
    "drafts": ([3000, 700, 2, 900], [4, 1, 5, 3], 2, 4, 32),
}


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,name", [("few_rows", n) for n in FEW] + [("many_rows", n) for n in ("short", "dealt", "halves")])
def test_bits_repeat_whatever_the_workspace_held_and_on_two_streams(rows, name, d):
    lens, new, h, share, page = (FEW if rows == "few_rows" else MANY)[name]
    kv, seqs, q, table, kv_lens, start = _problem(1500 + d, lens, new, h, share, d, page, BF16)
    assert _takes(kv, q, table) == rows
    x, qs = q.cuda(), torch.from_numpy(start).cuda()
    work = kv.attend_workspace(q.shape[0], q.shape[1], len(lens))
    first = None
    for fill in (0, 0xFF, 0x7C):
        work.fill_(fill)
        got = kv.attend(x, table, kv_lens, q_start=qs, return_lse=True, workspace=work)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    _check_each(*first, q, seqs, lens, start, BF16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    results = []
    for _ in range(4):
        for s in streams:
            results.append(kv.attend(x, table, kv_lens, q_start=qs, return_lse=True, stream=s))
    torch.cuda.synchronize()
    for got in results:
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,new,h,share", [([333, 20], [1, 1], 4, 2), ([700, 50, 0], [5, 3, 2], 2, 4),
                                              ([500, 130], [500, 130], 2, 8), ([1200, 600], [300, 600], 3, 4)])
def test_a_page_table_wider_than_the_sequences(lens, new, h, share, d):
    """As a captured step has it, for any later length: columns of no page, and of
    pages that are others'."""
    kv, seqs, q, table, kv_lens, start = _problem(1600 + d, lens, new, h, share, d, 32, F16)
    for fill in (-1, 0):
        wide = torch.full((len(lens), 1000), fill, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            wide[b, :-(-n // 32)] = table[b, :-(-n // 32)]
        out, lse = kv.attend(q.cuda(), wide, kv_lens, q_start=torch.from_numpy(start).cuda(), return_lse=True)
        _check_each(out, lse, q, seqs, lens, start, F16)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_strides_and_rows_left_alone(d):
    """q_start left out; q a slice of a fused projection, out heads first."""
    new, lens, h, share = 300, [450, 300, 304], 2, 4
    kv, seqs, q, table, kv_lens, start = _problem(1700 + d, lens, [new] * 3, h, share, d, 32, BF16)
    assert _takes(kv, q, table, ragged=False) == "many_rows"
    fused = torch.zeros(3 * new, 12, d, dtype=BF16, device="cuda")
    fused[:, 2:10] = q.cuda()
    around = torch.full((9, 3 * new, d), 3.0, dtype=BF16, device="cuda")
    kv.attend(fused[:, 2:10], table, kv_lens, out=around[:8].transpose(0, 1))
    _check_each(around[:8].transpose(0, 1), None, q, seqs, lens, start, BF16)
    assert (around[8] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_rows_captured_calls_follow_their_buffers(d):
    """A prompt's rows appended and attended over, captured once and replayed over
    other rows, lengths and pages."""
    rng = np.random.default_rng(d)
    h, share, page, most, batch = 2, 8, 16, 256, 2
    kv = dsq.KVCache(h, d, 64, page)
    k, v = (torch.zeros(batch * most, h, d, dtype=F16, device="cuda") for _ in range(2))
    q = torch.zeros(batch * most, h * share, d, dtype=F16, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    slots = torch.full((batch * most,), -1, dtype=torch.int64, device="cuda")
    table = torch.zeros(batch, 32, dtype=torch.int32, device="cuda")
    lens, start = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    work = kv.attend_workspace(q.shape[0], q.shape[1], batch)
    assert _takes(kv, q, table) == "many_rows"

    def step():
        kv.append(k, v, slots)
        kv.attend(q, table, lens, q_start=start, out=out, lse=lse, workspace=work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for new in ([256, 256], [30, 200], [0, 1], [129, 255]):
        x = torch.from_numpy(rng.standard_normal(tuple(q.shape))).half()
        rows = [_rows(rng, batch * most, h, d).half() for _ in range(2)]
        pages = rng.permutation(64).reshape(batch, 32)
        at, seqs, where = 0, [], np.full(batch * most, -1)
        for b, n in enumerate(new):
            t = np.arange(n)
            where[at:at + n] = pages[b, t // page] * page + t % page
            seqs.append(tuple(_held(r[at:at + n]) for r in rows))
            at += n
        for to, what in ((k, rows[0]), (v, rows[1]), (q, x), (slots, torch.from_numpy(where)), (table, torch.from_numpy(pages)),
                         (lens, torch.tensor(new)), (start, torch.tensor([0, new[0], sum(new)]))):
            to.copy_(what)
        out.fill_(3.0)
        g.replay()
        _check_each(out, lse, x, seqs, new, [0, new[0], sum(new)], F16)
        assert (out[sum(new):] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows,name", [("few_rows", "dealt"), ("many_rows", "dealt")])
def test_calls_that_follow_one_another_read_nothing_early(rows, name, d):
    """append, attend, read and attend again, launched early behind one another on one
    stream and one workspace, many times over: each call sees what the one before
    it wrote."""
    lens, new, h, share, page = (FEW if rows == "few_rows" else MANY)[name]
    kv, seqs, q, table, kv_lens, start = _problem(1800 + d, lens, new, h, share, d, page, F16)
    assert _takes(kv, q, table) == rows
    qs = torch.from_numpy(start).cuda()
    rng = np.random.default_rng(d)
    sets = []
    page0 = int(table[0, 0])
    slots = torch.arange(page, device="cuda") + page0 * page
    for i in range(2):   # two contents of the first page, two sets of queries
        k, v = (_rows(rng, page, h, d).half().cuda() for _ in range(2))
        sets.append((torch.randn(q.shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda").half(), k, v))
    work = kv.attend_workspace(q.shape[0], q.shape[1], len(lens))
    want = []
    for x, k, v in sets:
        kv.append(k, v, slots)
        torch.cuda.synchronize()
        out, lse = kv.attend(x, table, kv_lens, q_start=qs, return_lse=True, workspace=work)
        torch.cuda.synchronize()
        want.append((out, lse, *kv.read(slots)))
        torch.cuda.synchronize()
    outs = [(torch.zeros_like(q, device="cuda"), torch.zeros(q.shape[:2], device="cuda"),
             *(torch.zeros(page, h, d, dtype=F16, device="cuda") for _ in range(2))) for _ in range(20)]
    torch.cuda.synchronize()
    for i, (out, lse, k_out, v_out) in enumerate(outs):
        x, k, v = sets[i % 2]
        kv.append(k, v, slots)
        kv.attend(x, table, kv_lens, q_start=qs, out=out, lse=lse, workspace=work)
        kv.read(slots, k=k_out, v=v_out)
    torch.cuda.synchronize()
    for i, got in enumerate(outs):
        assert all(torch.equal(g, w) for g, w in zip(got, want[i % 2])), i


@pytest.mark.gpu
@pytest.mark.parametrize("bits,mode,batch", [(3, "affine", 1), (3, "affine", 2), (3, "affine", 16), (3, "lut", 1), (4, "lut", 1),
                                             (4, "lut", 3), (4, "lut", 8), (2, "bitplane", 1), (3, "bitplane", 4), (14, "intgrid", 1)])
def test_a_product_launched_early_behind_attention_reads_its_output(bits, mode, batch):
    """Attention lets the product behind it start while it still runs; the product's
    rows are the attention's all the same, bit for bit as after a synchronisation."""
    import synth
    h, heads, d, rows = 2, 8, 128, 512
    p = synth.make_problem(rows, heads * d, bits, mode, 0.01, "uniform", 3, 1)
    with dsq.Handle(dsq.pack_problem(p)) as mat:
        n = 20000 // batch
        kv, _, _, table, kv_lens, _ = _problem(1900, [n] * batch, [1] * batch, h, heads // h, d, 64, F16)
        qs = [torch.randn(batch, heads, d, generator=torch.Generator("cuda").manual_seed(i), device="cuda").half() for i in range(2)]
        work = kv.attend_workspace(batch, heads, batch)
        want = []
        for q in qs:
            out = kv.attend(q, table, kv_lens, workspace=work)
            torch.cuda.synchronize()
            want.append(mat.gemv(out.view(batch, heads * d)))
            torch.cuda.synchronize()
        out = torch.zeros(batch, heads, d, dtype=F16, device="cuda")
        ys = torch.zeros(20, batch, rows, dtype=F16, device="cuda")
        torch.cuda.synchronize()
        for i in range(20):
            kv.attend(qs[i % 2], table, kv_lens, out=out, workspace=work)
            mat.gemv(out.view(batch, heads * d), ys[i])
        torch.cuda.synchronize()
        for i in range(20):
            assert torch.equal(ys[i], want[i % 2]), i
        assert not torch.equal(want[0], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 3, 400])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attend_without_pages_or_columns(d, new):
    """No cache memory, no column of the page table, no token of any sequence."""
    q = torch.randn(2 * new, 8, d, device="cuda").half()
    lens = torch.tensor([5, 900], dtype=torch.int32, device="cuda")
    for pages, cols, n in ((0, 3, lens), (4, 0, lens), (0, 0, lens), (4, 3, lens * 0), (4, 3, -lens)):
        kv = dsq.KVCache(2, d, pages, 16)
        if pages:
            kv.data.fill_(0xFF)
        table = torch.zeros(2, cols, dtype=torch.int32, device="cuda")
        for start in (None, torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")):
            for causal in (True, False):
                out, lse = kv.attend(q, table, n, q_start=start, causal=causal, out=torch.ones_like(q), return_lse=True)
                assert not out.any() and torch.isneginf(lse).all()
    kv = dsq.KVCache(2, d, 4, 16)   # no sequence, no row
    none = kv.attend(q[:0], torch.zeros(0, 3, dtype=torch.int32, device="cuda"), lens[:0])
    assert none.shape == (0, 8, d)
    assert kv.attend(q[:0], torch.zeros(2, 3, dtype=torch.int32, device="cuda"), lens).shape == (0, 8, d)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [1, 5])
def test_attend_one_page_for_all_and_queries_shared_by_heads(new):
    """A page as large as the sequence, one kv head for 1500 query heads that are one
    and the same row in memory."""
    n, page, d = 3000, 4096, 64
    kv, seqs, q, table, kv_lens, start = _problem(1950, [n], [new], 1, 1, d, page, BF16, extra=0)
    heads = 1500
    out, lse = kv.attend(q.cuda().expand(new, heads, d), table, kv_lens, return_lse=True)
    # each within its bounds; not bit for bit alike, as the jobs' tokens are dealt out at different places
    _check_each(out, lse, q.expand(new, heads, d), seqs, [n], start, BF16)


@pytest.mark.gpu
def test_kernel_question_of_sizes_past_32_bits():
    kv = dsq.KVCache(2, 64, 4, 16)
    sizes = dict(q_tokens=400, q_heads=16, batch=1, table_pages=4)
    assert kv.attend_kernel(**sizes, window=(1 << 32) + 1) == kv.attend_kernel(**sizes, window=(1 << 31) - 1)
    for name, v in (("q_tokens", 1 << 64), ("q_heads", (1 << 32) + 16), ("batch", (1 << 32) + 1), ("table_pages", 1 << 32)):
        with pytest.raises(ValueError):
            kv.attend_kernel(**{**sizes, name: v})
    for change in (dict(window=-1), dict(window=3, causal=False), dict(q_heads=15)):
        with pytest.raises(dsq.DSQError) as e:
            kv.attend_kernel(**{**sizes, **change})
        assert e.value.status == BAD
