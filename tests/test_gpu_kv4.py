"""GPU checks of the 4-bit paged cache and of beam selection against their 64-bit definitions."""
import math

import numpy as np
import pytest

import kv4_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAGE = 64


@pytest.fixture(scope="module")
def kv4():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kv_cached_qwen3_gb300 import kv4
    return kv4


def dtype_of(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def rnd(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def shuffled(cache, seed):
    """The cache with its pages in another order."""
    g = torch.Generator().manual_seed(seed)
    cache.page_table.copy_(torch.randperm(cache.n_pages, generator=g)[:cache.page_table.numel()].view_as(cache.page_table))
    return cache


def edge_rows(x):
    """Blocks where a quantizer can go wrong, put into the first rows of x [..., 32 n]."""
    f = x.view(-1, 32)
    n = f.shape[0]
    vals = [torch.zeros(32), torch.full((32,), -0.0), torch.linspace(-1, 1, 32), torch.full((32,), 3.0),
            torch.arange(32.) - 16,                                           # ties of +m and -m, codes on borders
            torch.cat([torch.tensor([8., -8.]), torch.arange(30.) / 2 - 7.5]),   # exactly half way between codes
            torch.full((32,), 1e-40), torch.linspace(-3e-39, 3e-39, 32), torch.linspace(-1e-6, 1e-6, 32),
            torch.linspace(-6e5, 5e5, 32), torch.linspace(-3e38, 3e38, 32)]
    for i, v in enumerate(vals):
        if i < n:
            f[i] = v.to(x.dtype).to(x.device)
    return x


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("L,B,T,H,D,dt,order", [
    (1, 1, 1, 1, 64, "f32", "rows"), (1, 1, 1, 8, 128, "bf16", "rows"), (2, 3, 65, 3, 128, "f32", "rows"),
    (2, 3, 70, 2, 64, "bf16", "rows"), (3, 1, 130, 5, 128, "f32", "heads"), (1, 2, 9, 4, 128, "bf16", "packed"),
    (1, 2, 9, 4, 64, "f32", "odd"), (2, 3, 100, 3, 64, "bf16", "odd"), (1, 2, 131, 2, 64, "f32", "rows"),
    (1, 4, 200, 3, 128, "bf16", "packed"), (1, 2, 95, 2, 128, "f32", "rows"), (1, 2, 33, 2, 128, "bf16", "heads")])
def test_write_read(kv4, L, B, T, H, D, dt, order):
    dtype = dtype_of(dt)
    if order == "rows":
        kv = [rnd(s, L, B, T, H, D, dtype=dtype) for s in (1, 2)]
        for t in kv:
            edge_rows(t)
    elif order == "heads":      # as a state is exported: [layer][head][row]
        kv = [rnd(s, L, B, H, T, D, dtype=dtype).transpose(2, 3) for s in (1, 2)]
    else:                       # slices of a packed projection; "odd": heads off 16-byte boundaries
        extra = 0 if order == "packed" else 3
        x = rnd(1, L, B, T, 2 * H * D + extra, dtype=dtype)
        kv = [x[..., i * H * D + extra:(i + 1) * H * D + extra].unflatten(-1, (H, D)) for i in (0, 1)]
    c = shuffled(kv4.KV4Cache(B + 2, T + 100, L + 1, H, D), 3)
    start = torch.tensor([(37 * b) % 100 for b in range(B)], dtype=torch.int32).cuda()
    count = torch.tensor([max(0, T - 3 * b) for b in range(B)], dtype=torch.int32).cuda()
    c.write(kv[0], kv[1], start=start, count=count, layer0=1, stream0=2)
    out = [torch.full((L, B, T, H, D), 7.0, dtype=dtype, device="cuda") for _ in (0, 1)]
    c.read(*out, start=start, count=count, layer0=1, stream0=2)
    for t, o in zip(kv, out):
        x = host(t)
        want = torch.from_numpy(ref.q4_roundtrip(x)).to(dtype).double().numpy()   # exact in f32, rounded once to bf16
        for b in range(B):
            n = int(count[b])
            np.testing.assert_array_equal(host(o)[:, b, :n], want[:, b, :n])
            assert (host(o)[:, b, n:] == 7.0).all()
    # the stored bytes, by the layout's definition
    for pool, t, is_v in ((c.k, kv[0], False), (c.v, kv[1], True)):
        codes, d = ref.q4_quantize(host(t))
        s0 = int(start[0])
        for page in range(c.pages_per_stream):
            lo, hi = max(0, page * PAGE - s0), min(int(count[0]), (page + 1) * PAGE - s0)
            if lo >= hi:
                continue
            cc, dd = np.zeros((PAGE, D), np.uint8), np.zeros((PAGE, D // 32), np.float16)
            r0 = lo + s0 - page * PAGE
            cc[r0:r0 + hi - lo], dd[r0:r0 + hi - lo] = codes[L - 1, 0, lo:hi, H - 1], d[L - 1, 0, lo:hi, H - 1]
            got = pool[int(c.page_table[2, page]), L, H - 1].cpu().numpy()
            np.testing.assert_array_equal(got, ref.tile_bytes(cc, dd, is_v))
    assert c.sync_status() == 0
    assert not c.k[:, 0].any() and not c.v[:, 0].any()          # the other layer is untouched


def test_codes_on_borders_are_exact(kv4):
    """Values on and next to the borders between codes (f32 neighbours), for many maxima of both signs."""
    rng = np.random.default_rng(5)
    n = 512
    m = np.exp(rng.uniform(-60, 10, n)) * rng.choice([-1, 1], n)
    m = m.astype(np.float32).astype(np.float64)
    k = rng.integers(0, 17, (n, 32))
    x = ((17 - 2 * k) * m[:, None] / 16).astype(np.float32)
    step = rng.integers(-1, 2, (n, 32))
    x = np.where(step < 0, np.nextafter(x, -np.inf), np.where(step > 0, np.nextafter(x, np.inf), x))
    x = np.clip(x, -np.abs(m[:, None]), np.abs(m[:, None])).astype(np.float32)
    x[:, 0] = m
    t = torch.from_numpy(x.reshape(1, 1, n // 4, 1, 128)).cuda()
    c = kv4.KV4Cache(1, n // 4, 1, 1, 128)
    c.write(t, t)
    o = torch.empty_like(t)
    c.read(o, torch.empty_like(t))
    np.testing.assert_array_equal(host(o), ref.q4_roundtrip(host(t)))


@pytest.mark.parametrize("exponent", [0, -127, 90, 19])
def test_bf16_codes_are_exact(kv4, exponent):
    """Every pair of bf16 mantissas of a value and of its block's maximum, at exponents down to 2^-5 of it (near
    2^-127 some are subnormal, near 2^19 some maxima are clamped): many lie on a border between two codes."""
    mant = np.arange(128, 256) / 128.0
    x = np.stack(np.meshgrid(mant, mant, 2.0 ** np.arange(0, -6, -1), [1, -1], indexing="ij"), -1).reshape(128, -1, 4)
    x = x[..., 1] * x[..., 2] * x[..., 3]       # 1536 values for each maximum
    x = np.concatenate([x, x[:, :14]], 1).reshape(128, 50, 31)
    m = np.broadcast_to(mant[:, None, None] * np.where(np.arange(50) % 2, 1, -1)[None, :, None], (128, 50, 1))
    x = np.clip(x, -np.abs(m), np.abs(m))
    blocks = np.concatenate([m, x], -1).reshape(-1, 32) * 2.0 ** exponent
    t = torch.from_numpy(blocks.reshape(1, 1, -1, 1, 128)).to(torch.bfloat16).cuda()
    c = kv4.KV4Cache(1, t.shape[2], 1, 1, 128)
    c.write(t, t)
    codes, d = ref.q4_quantize(host(t)[0, 0, :, 0])
    for page in range(c.pages_per_stream):
        n = min(PAGE, t.shape[2] - page * PAGE)
        cc, dd = np.zeros((PAGE, 128), np.uint8), np.zeros((PAGE, 4), np.float16)
        cc[:n], dd[:n] = codes[page * PAGE:page * PAGE + n], d[page * PAGE:page * PAGE + n]
        np.testing.assert_array_equal(c.k[page, 0, 0].cpu().numpy(), ref.tile_bytes(cc, dd, False))
        np.testing.assert_array_equal(c.v[page, 0, 0].cpu().numpy(), ref.tile_bytes(cc, dd, True))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_blocks_of_zeros_and_of_both_signs(kv4, dt):
    """The largest magnitude with both signs, and zeros of both signs: the first one gives the scale its sign."""
    t = torch.zeros(1, 1, 8, 1, 128)
    t.view(8, 4, 32)[1::2, :, 0] = -0.0
    t.view(8, 4, 32)[2, :, 1:] = -0.0
    for i in range(4):
        t.view(8, 4, 32)[4 + i] = rnd(i, 4, 32).cpu().clamp(-1, 1)
        t.view(8, 4, 32)[4 + i, 0, [5, 20]] = torch.tensor([2.0, -2.0])
        t.view(8, 4, 32)[4 + i, 1, [7, 3]] = torch.tensor([2.0, -2.0])
        t.view(8, 4, 32)[4 + i, 2, [31, 8, 15]] = torch.tensor([2.0, -2.0, 2.0])
    t = t.to(dtype_of(dt)).cuda()
    for rows in (t, t.repeat(1, 1, 16, 1, 1)):       # by rows and by pages
        c = kv4.KV4Cache(1, rows.shape[2], 1, 1, 128)
        c.write(rows, rows)
        codes, d = ref.q4_quantize(host(rows)[0, 0, :PAGE, 0])
        n = len(codes)
        cc, dd = np.zeros((PAGE, 128), np.uint8), np.zeros((PAGE, 4), np.float16)
        cc[:n], dd[:n] = codes, d
        np.testing.assert_array_equal(c.k[0, 0, 0].cpu().numpy(), ref.tile_bytes(cc, dd, False))


def test_blocks_with_nan_or_inf_read_back_as_nan(kv4):
    t = rnd(1, 1, 1, 3, 2, 128)
    t[0, 0, 0, 0, 5] = float("nan")
    t[0, 0, 1, 1, 64] = float("inf")
    t[0, 0, 1, 1, 33] = -float("inf")
    c = kv4.KV4Cache(1, 64, 1, 2, 128)
    c.write(t, t)
    k, v = torch.empty_like(t), torch.empty_like(t)
    c.read(k, v)
    want = ref.q4_roundtrip(host(t))
    assert np.isnan(want).sum() == 96
    np.testing.assert_array_equal(host(k), want)
    np.testing.assert_array_equal(host(v), want)


def test_rows_outside_the_cache_are_skipped_and_reported(kv4):
    c = kv4.KV4Cache(2, 64, 1, 2, 64)
    t = rnd(1, 1, 2, 4, 2, 64)
    before = c.k.clone()
    start = torch.tensor([62, -3], dtype=torch.int32).cuda()
    c.write(t, t, start=start)
    out = torch.full_like(t, 9.0)
    c.read(out, out.clone(), start=start)
    want = ref.q4_roundtrip(host(t))
    np.testing.assert_array_equal(host(out)[0, 0, :2], want[0, 0, :2])     # positions 62, 63
    np.testing.assert_array_equal(host(out)[0, 1, 3], want[0, 1, 3])       # position 0
    assert (host(out)[0, 0, 2:] == 9).all() and (host(out)[0, 1, :3] == 9).all()
    assert c.sync_status() == 1 and c.sync_status() == 0
    c.k.copy_(before)
    c.page_table[0, 0] = 2      # n_pages
    c.page_table[1, 0] = -1
    c.write(t, t)
    assert torch.equal(c.k, before)
    assert c.sync_status() == 8


def test_pages_outside_the_cache_are_skipped_and_reported(kv4):
    """The same for enough rows that a page is written and read at once."""
    c = kv4.KV4Cache(3, 192, 1, 2, 128)
    t = rnd(1, 1, 3, 150, 2, 128)
    start = torch.tensor([100, -70, 10], dtype=torch.int32).cuda()
    c.page_table[2, 1] = 9      # n_pages
    before = c.k.clone()
    c.write(t, t, start=start)
    out = torch.full_like(t, 9.0)
    c.read(out, out.clone(), start=start)
    want = ref.q4_roundtrip(host(t))
    inside = np.zeros((3, 150), bool)
    inside[0, :92] = inside[1, 70:] = inside[2, :54] = inside[2, 118:] = True
    np.testing.assert_array_equal(host(out)[0][inside], want[0][inside])
    assert (host(out)[0][~inside] == 9).all()
    assert c.sync_status() == 9 and c.sync_status() == 0
    assert torch.equal(c.k[7], before[7])       # the page that stream 2 would have at its place


# ------------------------------------------------------------------ attention

def attend_tolerance(q, k, v, scale, dtype, want):
    """What f32 arithmetic may be off by. Scores: hd + 16 roundings of 2^-23 (products of two parts each, sums that
    may truncate) of scale * sum |q||k|, in both the numerator and the sum; probabilities in two fp16 parts and their
    exponentials: 2^-19; sums over n rows in chains of 16 rows a step: n / 16 + 64 roundings of 2^-23; all relative to
    the largest |v|. A bf16 result adds half a step, 2^-8 of the value."""
    if len(k) == 0:
        return 0.0
    g = q.shape[0] // k.shape[1]
    kmax = np.repeat(np.abs(k).max(0), g, axis=0)                            # [n_q, hd]
    s = scale * (np.abs(q) * kmax).sum(-1, keepdims=True)
    e = 2 * (q.shape[1] + 16) * 2.0 ** -23 * s + 2.0 ** -19 + (len(k) / 16 + 64) * 2.0 ** -23
    tol = e * np.abs(v).max()
    return tol + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0)


def filled(kv4, B, n, H, D, seed, layers=1, shuffle=True):
    """A cache with n rows in every stream, and the values they stand for [B, n, H, D] in f64 (of the last layer)."""
    c = kv4.KV4Cache(B, max(n, 1), layers, H, D)
    if shuffle:
        shuffled(c, seed)
    c.k.fill_(255)              # rows past a stream's length: NaN scales, which must not be read into a result
    c.v.fill_(255)
    if n:
        k, v = (rnd(seed + s, 1, B, n, H, D) for s in (1, 2))
        k[..., 3] *= 4          # a few dims stand out, as in real keys
        c.write(k, v, layer0=layers - 1)
        return c, ref.q4_roundtrip(host(k))[0], ref.q4_roundtrip(host(v))[0]
    return c, np.zeros((B, 0, H, D)), np.zeros((B, 0, H, D))


def check_attend(kv4, c, K, V, lens, H, G, D, dtype, fresh, scale=None, seed=50, max_len=None, layer=0, packed=False):
    B = len(lens)
    if packed:                  # q, k, v of the step as slices of one projection
        x = rnd(seed, B, (G + 2) * H * D, dtype=dtype)
        q, kn, vn = (t.unflatten(-1, (-1, D)) for t in x.split([G * H * D, H * D, H * D], -1))
    else:
        q, kn, vn = rnd(seed, B, H * G, D, dtype=dtype), rnd(seed + 1, B, H, D, dtype=dtype), rnd(seed + 2, B, H, D, dtype=dtype)
    out = c.attend(layer, q, torch.tensor(lens, dtype=torch.int32).cuda(), kn if fresh else None, vn if fresh else None,
                   scale=scale, max_len=max_len)
    assert out.dtype == dtype and out.shape == (B, H * G, D)
    got = host(out)
    scale = 1 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        k, v = K[b, :lens[b]], V[b, :lens[b]]
        if fresh:
            k, v = np.concatenate([k, host(kn)[b:b + 1]]), np.concatenate([v, host(vn)[b:b + 1]])
        want = ref.attend(host(q)[b], k, v, scale)
        tol = attend_tolerance(host(q)[b], k, v, scale, dtype, want)
        assert (np.abs(got[b] - want) <= tol).all(), (b, lens[b], np.abs(got[b] - want).max(), np.max(tol))
    return out


@pytest.mark.parametrize("lens", [[0], [1], [63, 64, 65], [0, 130, 1, 200], [1000, 7, 64, 0, 999]])
@pytest.mark.parametrize("H,G,D", [(1, 1, 64), (2, 2, 128), (3, 3, 64), (2, 5, 128), (1, 7, 64), (2, 8, 128), (4, 4, 128)])
@pytest.mark.parametrize("dt,fresh", [("f32", True), ("bf16", False)])
def test_attend(kv4, lens, H, G, D, dt, fresh):
    c, K, V = filled(kv4, len(lens), max(lens), H, D, 11)
    check_attend(kv4, c, K, V, lens, H, G, D, dtype_of(dt), fresh)
    assert c.sync_status() == 0


@pytest.mark.parametrize("n,B,H,G,D", [(5001, 2, 2, 2, 128), (9000, 1, 1, 8, 64), (2111, 9, 3, 4, 128)])
def test_attend_long(kv4, n, B, H, G, D):
    c, K, V = filled(kv4, B, n, H, D, 12, layers=2)
    lens = [n] + [n * (b + 1) // (B + 1) for b in range(B - 1)]
    outs = [check_attend(kv4, c, K, V, lens, H, G, D, torch.float32, False, layer=1, max_len=m) for m in (None, 1, n)]
    # the same bits twice: nothing depends on an order of arrival
    again = check_attend(kv4, c, K, V, lens, H, G, D, torch.float32, False, layer=1, max_len=n)
    assert torch.equal(outs[2], again)


@pytest.mark.parametrize("G,dt,fresh", [(1, "bf16", True), (2, "f32", False), (4, "f32", True), (8, "bf16", False),
                                        (8, "f32", True)])
def test_attend_many_streams(kv4, G, dt, fresh):
    """More work than a wave of CTAs, of very different lengths: ranges that hold many rows, and parts of rows."""
    B, n, H, D = 40, 1000, 8, 128
    c, K, V = filled(kv4, B, n, H, D, 14)
    rng = np.random.default_rng(G)
    lens = [int(x) for x in rng.integers(0, n + 1, B)]
    lens[:6] = [0, 1, 64, n, 0, 63]
    lens[-1] = 0
    outs = [check_attend(kv4, c, K, V, lens, H, G, D, dtype_of(dt), fresh) for _ in range(2)]
    assert torch.equal(outs[0], outs[1])
    check_attend(kv4, c, K, V, [n] * B, H, G, D, dtype_of(dt), fresh)
    assert c.sync_status() == 0
    # a page that is not there, and a length past the pages: those streams alone are told apart
    c.page_table[3, 2] = c.n_pages
    lens[7] = 16 * PAGE + 1
    q = rnd(60, B, H * G, D, dtype=dtype_of(dt))
    got = host(c.attend(0, q, torch.tensor(lens, dtype=torch.int32).cuda()))
    for b in (2, 3, 7, 8):
        keep = np.r_[0:128, 192:n] if b == 3 else np.arange(0 if b == 7 else lens[b])
        want = ref.attend(host(q)[b], K[b, keep], V[b, keep], D ** -0.5)
        tol = attend_tolerance(host(q)[b], K[b, keep], V[b, keep], D ** -0.5, dtype_of(dt), want)
        assert (np.abs(got[b] - want) <= tol).all(), b
    assert c.sync_status() == 9


def test_attend_packed_rows_and_scales(kv4):
    c, K, V = filled(kv4, 3, 100, 2, 128, 13)
    check_attend(kv4, c, K, V, [100, 64, 5], 2, 3, 128, torch.bfloat16, True, packed=True)
    check_attend(kv4, c, K, V, [100, 64, 5], 2, 3, 128, torch.float32, True, scale=2.0, packed=True)   # peaked rows
    check_attend(kv4, c, K, V, [100, 64, 5], 2, 3, 128, torch.float32, False, scale=0.0)               # plain means


@pytest.mark.parametrize("kmag,vmag", [(1e-3, 1e-6), (300.0, 1e4), (1e-7, 3e5)])
def test_attend_magnitudes(kv4, kmag, vmag):
    """Keys and values far from 1: the parts in fp16 are taken relative to the largest."""
    c = kv4.KV4Cache(2, 200, 1, 2, 128)
    k, v = rnd(1, 1, 2, 200, 2, 128) * kmag, rnd(2, 1, 2, 200, 2, 128) * vmag
    v[:, :, :40] *= 1e-3        # small values first, then large ones
    c.write(k, v)
    check_attend(kv4, c, ref.q4_roundtrip(host(k))[0], ref.q4_roundtrip(host(v))[0], [200, 33], 2, 2, 128,
                 torch.float32, False, scale=0.3 / kmag / math.sqrt(128))


def test_attend_nan_blocks_stay_in_their_place(kv4):
    """A NaN key makes its heads' rows NaN, a NaN value block its dims; past the length neither is seen."""
    c = kv4.KV4Cache(2, 70, 1, 2, 128)
    k, v = rnd(1, 1, 2, 70, 2, 128), rnd(2, 1, 2, 70, 2, 128)
    v[0, 0, 3, 0, 40] = float("nan")
    k[0, 1, 68, 1, 0] = float("inf")
    c.write(k, v)
    K, V = ref.q4_roundtrip(host(k))[0], ref.q4_roundtrip(host(v))[0]
    q = rnd(3, 2, 4, 128)
    for lens in ([70, 70], [3, 68]):
        got = host(c.attend(0, q, torch.tensor(lens, dtype=torch.int32).cuda()))
        for b in range(2):
            want = ref.attend(host(q)[b], K[b, :lens[b]], V[b, :lens[b]], 1 / math.sqrt(128))
            np.testing.assert_array_equal(np.isnan(got[b]), np.isnan(want))
    assert not np.isnan(got).any()


def test_attend_bad_lengths_and_pages(kv4):
    c, K, V = filled(kv4, 3, 130, 2, 64, 14)
    q = rnd(3, 3, 4, 64)
    lens = torch.tensor([-1, 193, 130], dtype=torch.int32).cuda()    # three pages a stream: 192 positions
    good = c.attend(0, q, torch.tensor([130, 130, 130], dtype=torch.int32).cuda())
    assert c.sync_status() == 0
    out = c.attend(0, q, lens, k_new=rnd(4, 3, 2, 64), v_new=rnd(5, 3, 2, 64))
    assert not out[:2].any() and c.sync_status() == 1
    c.page_table[2, 1] = c.n_pages
    out = c.attend(0, q, torch.tensor([130, 130, 130], dtype=torch.int32).cuda())
    assert torch.equal(out[:2], good[:2]) and c.sync_status() == 8
    keep = np.r_[0:64, 128:130]                                      # the bad page's keys are not attended
    want = ref.attend(host(q)[2], K[2, keep], V[2, keep], 1 / 8)
    assert np.abs(host(out)[2] - want).max() < 1e-4


def test_attend_where_streams_share_pages(kv4):
    """One page named by several streams and twice by one, as after reordering or for a common prompt."""
    c, K, V = filled(kv4, 3, 128, 2, 128, 15, shuffle=False)
    c.page_table.copy_(torch.tensor([[0, 1], [0, 3], [4, 4]], dtype=torch.int32))
    K = np.stack([K[0], np.concatenate([K[0, :64], K[1, 64:]]), np.concatenate([K[2, :64], K[2, :64]])])
    V = np.stack([V[0], np.concatenate([V[0, :64], V[1, 64:]]), np.concatenate([V[2, :64], V[2, :64]])])
    check_attend(kv4, c, K, V, [128, 100, 127], 2, 2, 128, torch.float32, True)
    assert c.sync_status() == 0


def test_attend_strided_queries_and_given_output(kv4):
    c, K, V = filled(kv4, 2, 90, 2, 64, 16)
    lens = torch.tensor([90, 33], dtype=torch.int32).cuda()
    wide = rnd(3, 2, 6, 2, 64)
    base = c.attend(0, wide[:, :, 0].contiguous(), lens)
    out = torch.full((2, 6, 64), 5.0, device="cuda")
    assert c.attend(0, wide[:, :, 0], lens, out=out) is out and torch.equal(out, base)
    off = torch.empty(2 * 6 * 64 + 1, device="cuda")[1:].view(2, 6, 64)     # off 16-byte boundaries
    off.copy_(wide[:, :, 0])
    assert torch.equal(c.attend(0, off, lens), base)
    assert c.attend(0, wide[:0, :, 0], lens[:0]).shape == (0, 6, 64)
    neg = c.attend(0, wide[:, :, 0], lens, scale=-0.3)                       # a negative scale is a scale
    for b in range(2):
        n = int(lens[b])
        want = ref.attend(host(wide[:, :, 0])[b], K[b, :n], V[b, :n], -0.3)
        tol = attend_tolerance(host(wide[:, :, 0])[b], K[b, :n], V[b, :n], 0.3, torch.float32, want)
        assert (np.abs(host(neg)[b] - want) <= tol).all()


# ------------------------------------------------------------------ selection

def check_select(logits, scores, ended=None, eos=-1):
    from kv_cached_qwen3_gb300.beam import beam_select
    tok, par, best, done = (t.cpu().numpy() for t in beam_select(logits, scores, ended=ended, eos_id=eos))
    S, W, V = logits.shape
    for i in range(S):
        t, p, s, d = ref.beam_select(host(logits)[i], host(scores)[i], None if ended is None else ended[i].cpu().numpy(), eos)
        np.testing.assert_array_equal(tok[i], t)
        np.testing.assert_array_equal(par[i], i * W + p)
        np.testing.assert_array_equal(done[i] != 0, d)
        # a score: the logarithm of a sum of V terms (its exponentials within 2 units, pairs summed over at most
        # V / 32 + 32 roundings) and two roundings of values up to |s|
        fin = np.isfinite(s)
        np.testing.assert_array_equal(best[i][~fin], s[~fin])
        got, s = best[i][fin], s[fin]
        assert (np.abs(got - s) <= (V / 32 + 40) * 2.0 ** -24 + 2.0 ** -23 * np.abs(s)).all()


@pytest.mark.parametrize("S,W,V,dt", [(1, 1, 1, "f32"), (1, 1, 5, "bf16"), (2, 4, 4, "f32"), (3, 5, 257, "bf16"),
                                      (1, 32, 33, "f32"), (2, 32, 4099, "f32"), (5, 3, 50021, "bf16"),
                                      (1, 8, 151669, "f32"), (40, 2, 1000, "f32"), (1, 32, 32003, "f32"),
                                      (3, 17, 20000, "bf16"), (2, 32, 9001, "f32"), (1, 31, 600, "bf16")])
def test_select(kv4, S, W, V, dt):
    x = (rnd(1, S, W, V) * 2).to(dtype_of(dt))
    scores = -10 * rnd(2, S, W).abs()
    check_select(x, scores)
    ended = (rnd(3, S, W) > 0.5).to(torch.int32)
    check_select(x, scores, ended, V // 2)
    check_select(x, scores, torch.ones_like(ended), V - 1)


def test_select_ties_masks_and_specials(kv4):
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x = torch.zeros(1, 4, 300).cuda()
    check_select(x, torch.zeros(1, 4).cuda())                                  # every candidate is equal
    x[0, :, ::2] = -0.0
    check_select(x, torch.zeros(1, 4).cuda())                                  # -0 and 0 are
    first = torch.tensor([[0.0, -inf, -inf, low]]).cuda()                      # a search's first step
    check_select(rnd(1, 1, 4, 300), first)
    check_select(rnd(1, 1, 4, 300), torch.full((1, 4), -inf).cuda())           # nothing is left
    check_select(rnd(1, 1, 4, 300), torch.tensor([[float("nan"), inf, -3.0, 2.0]]).cuda())
    x = torch.full((1, 4, 300), -inf).cuda()
    check_select(x, torch.zeros(1, 4).cuda())                                  # every token is masked
    x[0, 2, 17] = 1.0
    x[0, 1, 299] = low
    check_select(x, -torch.arange(4.0)[None].cuda())                           # one candidate, then masked ones in order
    x = rnd(4, 1, 4, 300)
    x[0, 0, 5] = float("nan")
    x[0, 1, 6] = inf
    x[0, 2, 40:] = low
    check_select(x, torch.zeros(1, 4).cuda())
    check_select(x, first, torch.tensor([[0, 1, 0, 1]], dtype=torch.int32).cuda(), 299)


@pytest.mark.parametrize("V,dt", [(20000, "f32"), (20000, "bf16"), (40003, "f32"), (40003, "bf16")])
def test_select_long_masked_rows(kv4, V, dt):
    """Masked values (NaN, -inf, the type's lowest) between, before and after a row's logits, and rows of nothing else;
    40003: by parts over the whole GPU."""
    dtype = dtype_of(dt)
    low = torch.finfo(dtype).min
    x = (rnd(1, 3, 5, V) * 2).to(dtype)
    some = rnd(2, V) > 1
    x[0, 0, some] = float("nan")
    x[0, 1, : V - 700] = -float("inf")
    x[0, 2, 900:] = low
    x[0, 3, :] = float("nan")
    x[0, 4, some] = low
    x[1, :, : V // 2] = low
    x[1, 1] = low
    x[1, 2, some] = -float("inf")
    x[2] = -float("inf")            # fewer than five candidates in all
    x[2, 1, V - 2] = 3.0
    x[2, 4, 11] = 1.0
    check_select(x, -10 * rnd(3, 3, 5).abs())


def test_rows_past_four_gigabytes(kv4):
    """Pages whose bytes lie more than 2^32 from the pool's first."""
    L, H, D = 28, 8, 128
    n = 4300
    k = torch.empty(n, L, H, 36 * D, dtype=torch.uint8, device="cuda")
    assert k.numel() > 2 ** 32
    c = kv4.KV4Cache.over(k, torch.empty_like(k), torch.tensor([[n - 1, 3], [n - 2, n - 3]], dtype=torch.int32).cuda(), D)
    for T in (5, 128):
        kv = [rnd(s, 2, 2, T, H, D) for s in (1, 2)]
        c.write(kv[0], kv[1], layer0=L - 2)
        out = [torch.empty_like(t) for t in kv]
        c.read(*out, layer0=L - 2)
        for t, o in zip(kv, out):
            np.testing.assert_array_equal(host(o), ref.q4_roundtrip(host(t)))
    q = rnd(3, 2, 2 * H, D)
    got = host(c.attend(L - 1, q, torch.full((2,), 128, dtype=torch.int32).cuda()))
    K, V = (ref.q4_roundtrip(host(t))[1] for t in kv)
    for b in range(2):
        want = ref.attend(host(q)[b], K[b], V[b], D ** -0.5)
        assert (np.abs(got[b] - want) <= attend_tolerance(host(q)[b], K[b], V[b], D ** -0.5, torch.float32, want)).all()


def test_select_strided_rows(kv4):
    x = rnd(1, 2, 3, 515)
    check_select(x[..., 1:500], -rnd(2, 2, 3).abs())
    check_select(x[..., 3:].to(torch.bfloat16), -rnd(2, 2, 3).abs())
    check_select(x.transpose(0, 1), -rnd(2, 3, 2).abs())


# ------------------------------------------------------------------ reordering

def contents(c, lens):
    """Every stream's rows [layers, rows, heads, dims], K and V."""
    n = c.pages_per_stream * PAGE
    k = torch.zeros(c.n_layers, c.n_streams, n, c.n_kv_heads, c.head_dim, device="cuda")
    v = torch.zeros_like(k)
    c.read(k, v, count=lens)
    return [(k[:, s, :int(lens[s])].cpu(), v[:, s, :int(lens[s])].cpu()) for s in range(c.n_streams)]


def same(a, b):
    return all(torch.equal(x, y) for p, q in zip(a, b) for x, y in zip(p, q))


def writable_pages_are_owned(c, lens):
    t = c.page_table.cpu()
    n, pps = t.shape
    assert ((t - torch.arange(pps)) % pps == 0).all()
    for j in range(pps):
        for s in range(n):
            if int(lens[s]) // PAGE <= j:
                assert (t[:, j] == t[s, j]).sum() == 1, (s, j)


@pytest.mark.parametrize("n,lens", [(1, [70]), (4, [130] * 4), (5, [0, 64, 65, 192, 100]), (40, [100] * 40), (70, None)])
@pytest.mark.parametrize("R", [None, 3])
def test_reorder(kv4, n, lens, R):
    g = torch.Generator().manual_seed(n)
    if lens is None:
        lens = torch.randint(0, 193, (n,), generator=g).tolist()
    R = n if R is None else min(R, n)
    c = kv4.KV4Cache(n, 190, 2, 2, 64)
    k, v = rnd(1, 2, n, 192, 2, 64), rnd(2, 2, n, 192, 2, 64)
    at = torch.tensor(lens, dtype=torch.int32).cuda()
    c.write(k, v, count=at)
    for turn in range(4):
        old = contents(c, at)
        hi = n if turn < 3 else max(1, n // 3)         # the last turn: few survivors
        parents = torch.randint(0, hi, (R,), generator=g).to(torch.int32).cuda()
        full = torch.cat([parents.cpu(), torch.arange(R, n, dtype=torch.int32)])
        d, new = c.reorder(parents, at)
        assert torch.equal(new.cpu(), at.cpu()[full.long()])
        assert same(contents(d, new), [old[p] for p in full.tolist()])
        writable_pages_are_owned(d, new)
        d2, new2 = c.reorder(parents, at)              # again, from the old table
        assert torch.equal(d2.page_table, d.page_table) and same(contents(d2, new2), [old[p] for p in full.tolist()])
        c, at = d, new
        # the next row of every stream that has room goes to a page of its own
        room = (at < c.pages_per_stream * PAGE).to(torch.int32)
        row = [rnd(10 + turn + s, 2, n, 1, 2, 64) for s in (0, 100)]
        before = contents(c, at)
        c.write(*row, start=at, count=room)
        assert same(contents(c, at), before)
        at = at + room
    assert c.sync_status() == 0


@pytest.mark.parametrize("cut", [[150, 70, 64, 10], [0, 0, 0, 0], [130, 130, 130, 5]])
def test_reorder_after_streams_were_cut(kv4, cut):
    """Streams that share pages and are cut inside them get pages of their own again, all at once."""
    c = kv4.KV4Cache(4, 192, 2, 2, 64)
    k, v = rnd(1, 2, 4, 160, 2, 64), rnd(2, 2, 4, 160, 2, 64)
    c.write(k, v)
    at = torch.full((4,), 160, dtype=torch.int32).cuda()
    c, at = c.reorder(torch.tensor([2, 2, 2, 1], dtype=torch.int32).cuda(), at)
    old = contents(c, at)
    at = torch.minimum(at, torch.tensor(cut, dtype=torch.int32).cuda())
    want = [tuple(x[:, :n] for x in old[i]) for i, n in enumerate(cut)]
    d, new = c.reorder(torch.zeros(0, dtype=torch.int32).cuda(), at)      # R = 0: every stream stays
    assert new.tolist() == cut
    writable_pages_are_owned(d, new)
    assert same(contents(d, new), want)
    row = [rnd(20 + s, 2, 4, 30, 2, 64) for s in (0, 1)]
    d.write(*row, start=new)
    assert same(contents(d, new), want)
    assert d.sync_status() == 0


def test_reorder_reports_bad_values(kv4):
    c = kv4.KV4Cache(3, 64, 1, 1, 64)
    k = rnd(1, 1, 3, 10, 1, 64)
    c.write(k, k)
    at = torch.tensor([10, 10, 10], dtype=torch.int32).cuda()
    old = contents(c, at)
    d, new = c.reorder(torch.tensor([1, 3, -1], dtype=torch.int32).cuda(), at)
    assert same(contents(d, new), [old[1], old[1], old[2]]) and c.sync_status() == 8
    d, new = c.reorder(torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), torch.tensor([10, 65, -1], dtype=torch.int32).cuda())
    assert new.tolist() == [10, 64, 0] and c.sync_status() == 1


# ------------------------------------------------------------------ together

def test_beam_search_together(kv4):
    """A search as a program runs it: write the step's rows, attend, choose, reorder. Every step's attention is checked
    against rows kept dense and gathered by the chosen parents."""
    from kv_cached_qwen3_gb300.beam import beam_select
    S, W, H, G, D, V, n0 = 2, 3, 2, 2, 128, 97, 60
    N = S * W
    c = kv4.KV4Cache(N, 128, 1, H, D)
    k, v = rnd(1, 1, N, n0, H, D), rnd(2, 1, N, n0, H, D)
    c.write(k, v)
    K, V_ = ref.q4_roundtrip(host(k))[0], ref.q4_roundtrip(host(v))[0]
    lens = torch.full((N,), n0, dtype=torch.int32).cuda()
    head = rnd(3, H * G * D, V) / 8
    scores = torch.tensor([[0.0] + [float("-inf")] * (W - 1)] * S).cuda()
    ended = torch.zeros(S, W, dtype=torch.int32).cuda()
    for t in range(40):
        q, kn, vn = rnd(100 + t, N, H * G, D), rnd(200 + t, N, H, D), rnd(300 + t, N, H, D)
        out = check_attend(kv4, c, K, V_, [n0 + t] * N, H, G, D, torch.float32, True, seed=400 + t)
        out = c.attend(0, q, lens, kn, vn)
        c.write(kn[None, :, None], vn[None, :, None], start=lens)
        K = np.concatenate([K, ref.q4_roundtrip(host(kn))[:, None]], 1)
        V_ = np.concatenate([V_, ref.q4_roundtrip(host(vn))[:, None]], 1)
        lens = lens + 1
        logits = (out.flatten(1) @ head).view(S, W, V)
        check_select(logits, scores, ended, 7)
        tok, par, scores, ended = beam_select(logits, scores, ended=ended, eos_id=7)
        c, lens = c.reorder(par.flatten(), lens)
        p = par.flatten().cpu().numpy()
        K, V_ = K[p], V_[p]
    assert c.sync_status() == 0


def test_captured_and_replayed_on_another_stream(kv4):
    """One step captured into two graphs, replayed at once on two streams with new inputs: each has its own scratch."""
    from kv_cached_qwen3_gb300.beam import beam_select
    sets = []
    for i in range(2):
        c, K, V = filled(kv4, 4, 700, 2, 128, 20 + i, shuffle=False)
        s = dict(c=c, K=K, V=V, pools=(c.k.clone(), c.v.clone()), q=rnd(1, 4, 4, 128), lens=torch.full((4,), 700, dtype=torch.int32).cuda(),
                 x=rnd(2, 1, 4, 5000), scores=-rnd(3, 1, 4).abs(), stream=torch.cuda.Stream())

        def step(s=s):
            s["out"] = s["c"].attend(0, s["q"], s["lens"], max_len=700)
            s["sel"] = beam_select(s["x"], s["scores"])
            s["new"], s["lens2"] = s["c"].reorder(s["sel"][1].flatten(), s["lens"])
        s["stream"].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s["stream"]):
            step()
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            step()
        sets.append(s)
    for rep in range(3):
        for i, s in enumerate(sets):
            s["q"].copy_(rnd(50 + 10 * rep + i, 4, 4, 128))
            s["x"].copy_(rnd(51 + 10 * rep + i, 1, 4, 5000))
            s["c"].k.copy_(s["pools"][0])       # streams given up in the last round hold others' rows
            s["c"].v.copy_(s["pools"][1])
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in sets:
            for b in range(4):
                want = ref.attend(host(s["q"])[b], s["K"][b], s["V"][b], 1 / math.sqrt(128))
                tol = attend_tolerance(host(s["q"])[b], s["K"][b], s["V"][b], 1 / math.sqrt(128), torch.float32, want)
                assert (np.abs(host(s["out"])[b] - want) <= tol).all()
            t, p, sc, _ = ref.beam_select(host(s["x"])[0], host(s["scores"])[0], None, -1)
            np.testing.assert_array_equal(s["sel"][0][0].cpu().numpy(), t)
            np.testing.assert_array_equal(s["sel"][1][0].cpu().numpy(), p)
            old = contents(s["c"], s["lens"])
            assert same(contents(s["new"], s["lens2"]), [old[j] for j in p])


def test_wrapper_refusals(kv4):
    from kv_cached_qwen3_gb300.beam import beam_select
    from kv_cached_qwen3_gb300.talker import TalkerError
    c = kv4.KV4Cache(2, 64, 1, 2, 64)
    q, lens = rnd(1, 2, 4, 64), torch.tensor([1, 1], dtype=torch.int32).cuda()
    for bad in (q.half(), q[..., :32], q[:, :3], rnd(1, 3, 4, 64), rnd(1, 2, 18, 64), q.cpu()):
        with pytest.raises(ValueError):
            c.attend(0, bad, lens)
    for kw in (dict(lens=lens.long()), dict(lens=lens[:1]), dict(lens=lens, k_new=rnd(1, 2, 2, 64)),
               dict(lens=lens, out=torch.empty(2, 4, 64).cuda().bfloat16())):
        with pytest.raises(ValueError):
            c.attend(0, q, **kw)
    with pytest.raises(TalkerError):
        c.attend(1, q, lens)
    x = rnd(1, 1, 2, 3, 2, 64)
    for a, b in ((x, x.bfloat16()), (x.half(), x.half()), (x[..., :32], x[..., :32]), (x, x[:, :, :2]),
                 (x[..., ::2], x[..., ::2])):
        with pytest.raises(ValueError):
            c.write(a, b)
    with pytest.raises(ValueError):
        c.write(x, x, start=torch.tensor([0], dtype=torch.int32).cuda())
    for kw in (dict(layer0=1), dict(stream0=1), dict(layer0=-1)):
        with pytest.raises(TalkerError):
            c.write(x, x, **kw)
    with pytest.raises(TalkerError):
        c.reorder(lens, lens, lens_out=lens)
    with pytest.raises(TalkerError):
        c.reorder(lens, lens, table_out=c.page_table)
    with pytest.raises(ValueError):
        c.reorder(lens, lens[:1])
    for bad in (lambda: kv4.KV4Cache(1, 64, 1, 1, 32), lambda: kv4.KV4Cache(0, 64, 1, 1, 64),
                lambda: kv4.KV4Cache.over(c.k, c.v[:1], c.page_table, 64), lambda: kv4.KV4Cache.over(c.k, c.v, c.page_table, 128),
                lambda: kv4.KV4Cache.over(c.k.cpu(), c.v.cpu(), c.page_table.cpu(), 64)):
        with pytest.raises(ValueError):
            bad()
    y, s = rnd(1, 1, 2, 10), torch.zeros(1, 2).cuda()
    for args, kw in (((y.half(), s), {}), ((y, s.double()), {}), ((y, s[:, :1]), {}), ((y, s), dict(eos_id=10)),
                     ((y, s), dict(ended=torch.zeros(1, 2, dtype=torch.int32).cuda())), ((y[..., :1], s), {}),
                     ((rnd(1, 1, 33, 40), torch.zeros(1, 33).cuda()), {})):
        with pytest.raises(ValueError):
            beam_select(*args, **kw)
