"""GPU checks of how many bits the attention over the 4-bit cache keeps: bounds follow the actual scores and
probabilities, and a bf16 result has to be one that the exact result, moved by that bound, rounds to."""
import math

import numpy as np
import pytest

import kv4_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def kv4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300 import kv4
    return kv4


def rnd(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def blocks(x):
    """The largest magnitude of each block of 32 dims, at every dim."""
    b = np.abs(x).reshape(x.shape[:-1] + (-1, 32))
    return np.broadcast_to(b.max(-1, keepdims=True), b.shape).reshape(x.shape)


def neighbours(x):
    """The magnitude of the even dim of each pair, at the odd one (0 at the even one)."""
    y = np.zeros_like(x)
    y[..., 1::2] = np.abs(x[..., ::2])
    return y


def attend_bound(q, k, v, scale, centred):
    """What the arithmetic of one stream may be off by: q [n_q, hd], k and v [n, n_kv, hd], at most 256 rows (a page
    a warp). One MMA adds 17 numbers, each cut 2^-24 of the largest at worst: 2^-20 of the sum of magnitudes.
    Scores: up to 4 such sums a block, q in two parts (2^-22), a few f32 roundings: 1.25 * 2^-18 of the sum of
    magnitudes, in which a code n of a block with scale d counts (n - 8) d where codes are centred (an odd dim's q
    meets its even neighbour's code too, at 2 / 16), n d and the offset 8 d else.
    Probabilities: exponents off by 2^-22 of the largest score and 2^-22 more, two parts 2^-20, sums of up to 96
    terms in f32 and 8 MMAs a dim (2^-20 each, the neighbour's at 2 / 16): 2^-16.5 in all, relative to p |v|; and half
    the least step of fp16, 2^-25, in the parts of every row's probability and of its product with a scale, where the
    largest probability is at least 2^6 and the block's largest scale brought to 2^2, by a factor of at most 2^15."""
    n, n_kv = k.shape[:2]
    g = q.shape[0] // n_kv
    qh = np.abs(q).reshape(n_kv, g, -1)
    size = np.abs(k) if centred else np.abs(k) + 2 * blocks(k)
    b = np.einsum("hgd,nhd->hgn", qh, size)
    if centred:
        b += np.einsum("hgd,nhd->hgn", qh, neighbours(k)) / 8
    s = np.einsum("hgd,nhd->hgn", q.reshape(n_kv, g, -1), k) * scale
    ds = 1.25 * 2.0 ** -18 * abs(scale) * b + 2.0 ** -22 * np.abs(s).max(-1, keepdims=True) + 2.0 ** -22
    p = np.exp(s - s.max(-1, keepdims=True))
    top = 1 / p.sum(-1, keepdims=True)
    p *= top
    size = np.abs(v) + neighbours(v) / 8
    e = p * (ds + (p * ds).sum(-1, keepdims=True) + 2.0 ** -16.5)
    most = blocks(v).max(0)[:, None]                            # 8 times the largest scale
    step = 2.0 ** -31 * (1 + 1 / np.clip(most / 8 * 2.0 ** 15, 2.0 ** -9, 4))
    out = np.einsum("hgn,nhd->hgd", e, size) + n * step * top * most
    return out.reshape(q.shape)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def check(got, q, k, v, scale, dtype):
    want = ref.attend(q, k, v, scale)
    tol = attend_bound(q, k, v, scale, dtype == torch.float32)
    if dtype == torch.float32:
        lo, hi = want - tol - U * np.abs(want), want + tol + U * np.abs(want)
    else:
        lo, hi = bf16(want - tol), bf16(want + tol)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (bad.sum(), got[bad][:4], want[bad][:4], tol[bad][:4])


def run(kv4, k, v, q, lens, scale, kn=None, vn=None):
    """k, v [B, n, H, D] written and attended; each stream checked."""
    B, n, H, D = k.shape
    c = kv4.KV4Cache(B, n, 1, H, D)
    c.write(k[None], v[None])
    K, V = ref.q4_roundtrip(host(k)), ref.q4_roundtrip(host(v))
    got = host(c.attend(0, q, torch.tensor(lens, dtype=torch.int32).cuda(), kn, vn, scale=scale))
    for b, m in enumerate(lens):
        kk, vv = K[b, :m], V[b, :m]
        if kn is not None:
            kk, vv = np.concatenate([kk, host(kn)[b:b + 1]]), np.concatenate([vv, host(vn)[b:b + 1]])
        check(got[b], host(q)[b], kk, vv, scale, q.dtype)
    assert c.sync_status() == 0


DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("H,G,D", [(2, 1, 64), (2, 2, 128), (1, 4, 128), (2, 5, 64), (3, 8, 128), (1, 7, 128)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("s", [0.05, 1.0, 4.0])
def test_random_rows(kv4, H, G, D, dt, s):
    lens = [1, 2, 3, 5, 64, 200]
    k, v = rnd(1, 6, 200, H, D), rnd(2, 6, 200, H, D)
    q = rnd(3, 6, H * G, D, dtype=DT[dt])
    run(kv4, k, v, q, lens, s / math.sqrt(D))
    kn, vn = rnd(4, 6, H, D, dtype=DT[dt]), rnd(5, 6, H, D, dtype=DT[dt])
    run(kv4, k, v, q, lens, s / math.sqrt(D), kn, vn)


@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("bits,mag", [(12, 1e-6), (15, 1e-5), (12, 1.0), (9, 1e-3)])
def test_one_key_above_many(kv4, G, dt, bits, mag):
    """One key whose probability is 2^bits times that of each other, whose values add up to much of the result."""
    n, D = 250, 128
    k = torch.zeros(1, n, 1, D)
    k[0, 7] = 1.0
    q = torch.ones(1, G, D)
    v = (1 + torch.rand(1, n, 1, D, generator=torch.Generator().manual_seed(1))) * mag
    v[0, 7] *= 2.0 ** -8
    run(kv4, k.cuda(), v.cuda(), q.to(DT[dt]).cuda(), [n], bits * math.log(2) / D)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("G", [1, 6])
@pytest.mark.parametrize("D", [64, 128])
def test_blocks_of_values_of_very_different_size(kv4, dt, G, D):
    """Each block of dims keeps its bits, whatever the others hold."""
    n = 150
    k, v = rnd(1, 2, n, 2, D), rnd(2, 2, n, 2, D)
    v[..., 32:64] *= 2.0 ** -13
    v[:, :, :, :32] *= 2.0 ** 12
    v[:, 100:, :, 32:64] *= 8      # larger ones come later
    run(kv4, k, v, rnd(3, 2, 2 * G, D, dtype=DT[dt]), [n, 101], 2 / math.sqrt(D))


@pytest.mark.parametrize("G,D", [(1, 64), (4, 128), (5, 128), (8, 64)])
def test_bf16_queries_are_exact(kv4, G, D):
    """Two keys whose exact scores are equal, one on even dims and one on odd ones, at a score of 100: values of
    opposite sign cancel. q has numbers whose sixteenths need all of bf16's bits beside them."""
    k = torch.zeros(1, 2, 1, D)
    k[0, 0, 0, ::2] = 1.0
    k[0, 1, 0, 1::2] = 1.0
    v = rnd(2, 1, 2, 1, D)
    v[0, 1] = -v[0, 0]
    v[0, :, :, ::32] = torch.tensor([4.0, -4.0]).view(2, 1, 1).cuda()
    for a in (255, 253, 251, 193, 129):
        q = torch.full((1, G, D), a / 128, dtype=torch.bfloat16)
        run(kv4, k.cuda(), v, q.cuda(), [2], 100 / (D / 2 * a / 128))


@pytest.mark.parametrize("H,G,D", [(2, 2, 128), (1, 3, 64), (2, 8, 128), (1, 5, 64)])
def test_f32_queries_with_bf16_results(kv4, H, G, D):
    """The form of a Talker's steps on the tensor cores: q keeps 22 bits. Each q is 1 + 2^-12 times one of bf16, which
    its first eleven bits would lose, at scores of up to 100 of two keys that nearly cancel."""
    k = torch.zeros(1, 2, H, D)
    k[0, 0, :, ::2] = 1.0
    k[0, 1, :, 1::2] = 1.0
    v = rnd(2, 1, 2, H, D)
    v[0, 1] = -v[0, 0]
    v[0, :, :, ::32] = torch.tensor([4.0, -4.0]).view(2, 1, 1).cuda()
    c = kv4.KV4Cache(1, 2, 1, H, D)
    c.write(k.cuda()[None], v[None])
    q = torch.full((1, H * G, D), 1.0)
    q[..., 1::2] = 1 + 2.0 ** -12
    q, lens = q.cuda(), torch.tensor([2], dtype=torch.int32).cuda()
    out = torch.empty(1, H * G, D, dtype=torch.bfloat16, device="cuda")
    scale = 100 / (D / 2)
    kv4.launch(c.device.index, c._lib.talker_test_kv4_attend_mixed, "talker_test_kv4_attend_mixed", c._ref, 1, lens.data_ptr(),
               2, H * G, scale, q.data_ptr(), out.data_ptr(), None, 0)
    check(host(out)[0], host(q)[0], ref.q4_roundtrip(host(k))[0], ref.q4_roundtrip(host(v))[0], scale, torch.bfloat16)


@pytest.mark.parametrize("G,D", [(2, 128), (8, 128), (3, 64), (6, 64)])
def test_long_rows_do_not_shrink(kv4, G, D):
    """Values of one sign over a row that one CTA attends (max_len says it is short): rounded sums leave errors of either
    sign, so their mean over all dims stays at what the chains of two MMAs cut off, 2^-24 each, and the parts' own last
    bits. Sums cut off from start to end would be 313 * 2^-25 low and more."""
    n = 20000
    c = kv4.KV4Cache(1, n, 1, 1, D)
    k, v = rnd(1, 1, 1, n, 1, D), 1 + torch.rand(1, 1, n, 1, D, generator=torch.Generator().manual_seed(2)).cuda()
    c.write(k, v)
    q = rnd(3, 1, G, D)
    got = host(c.attend(0, q, torch.tensor([n], dtype=torch.int32).cuda(), max_len=1))[0]
    want = ref.attend(host(q)[0], ref.q4_roundtrip(host(k))[0, 0], ref.q4_roundtrip(host(v))[0, 0], D ** -0.5)
    e = (got - want) / want
    assert abs(e.mean()) <= 2.0 ** -21 and np.abs(e).max() <= 2.0 ** -18, (e.mean(), np.abs(e).max())
