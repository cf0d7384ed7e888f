"""GPU: residual RMSNorm, rotary positions and 4-bit products against 64 bits."""
import math

import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
F64 = torch.float64
STEP = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def assert_within(got, want, bound):
    got, want = got.double().cpu(), want.double()
    ok = (got - want).abs() <= bound
    assert ok.all(), (got[~ok][:4], want[~ok][:4], (bound.expand_as(ok) if torch.is_tensor(bound) else bound))


# ------------------------------------------------------------------ norm

def check_norm(x, gain, res, out, block=0, eps=1e-6, into=None):
    """y: the mean of squares is a sum of `width` f32 terms whose roundings follow one another at most 8 times in a thread's
    vector, twice per thread and ten times across threads, or chunk after chunk in rows past 16384 values; s, the root, the
    division and two products round a few times more."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    width = x.shape[-1]
    y, s, scales = rms_norm(x, gain, eps=eps, residual=res, out_dtype=DT[out], block=block, out=into)
    want, total = ref.rms_norm(x.cpu(), gain.cpu(), eps, None if res is None else res.cpu())
    near = (32 + width / 8192) * STEP
    if res is not None:
        assert_within(s, total, total.abs() * (ref.half_step(s.dtype) + STEP * (s.dtype is not torch.float32)) + 1e-45)
    else:
        assert s is None
    if out != "e4m3":
        assert scales is None
        assert_within(y, want, want.abs() * (near + ref.half_step(y.dtype) * (1 + near) * (out != "f32")) + 1e-37)
        return y
    assert scales.shape == x.shape[:-1] + (-(-width // block) if block else 1,)
    tops = torch.stack([want[..., j:j + (block or width)].abs().amax(-1) for j in range(0, width, block or width)], -1)
    assert_within(scales, tops / 448, tops / 448 * near)
    spread = ref.by_block(scales.double().cpu(), block, width)
    # half a step of three bits and the leading one, or of the smallest steps, 2^-9
    assert_within(y.float().cpu().double() * spread, want, want.abs() * (2.0 ** -4 + 4 * near) + spread * 2.0 ** -10 * (1 + near))
    return y


@pytest.mark.parametrize("x,res,out,block", [("f32", "f32", "f32", 0), ("f32", None, "bf16", 0), ("bf16", "f32", "e4m3", 32), ("bf16", "bf16", "bf16", 0),
                                             ("f32", "bf16", "e4m3", 64), ("bf16", None, "f32", 0), ("bf16", "f32", "e4m3", 128), ("f32", None, "e4m3", 0)])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 32), (2, 33), (130, 128), (7, 255), (3, 1000), (1, 1024), (9, 5120), (2, 8191), (2, 8200), (1, 16384),
                                        (2, 16389), (1, 40003)])
def test_norm(x, res, out, block, rows, width):
    xs = (ref.rnd(1, rows, width) * 2).to(DT[x]).cuda()
    r = None if res is None else (ref.rnd(2, rows, width) * 5).to(DT[res]).cuda()
    check_norm(xs, (1 + 0.1 * ref.rnd(3, width)).cuda(), r, out, block)


@pytest.mark.parametrize("x,res,out,block,rows,width", [
    ("f32", "f32", "bf16", 0, 80003, 13), ("bf16", "bf16", "bf16", 0, 80003, 47), ("bf16", "f32", "e4m3", 0, 40009, 65), ("f32", "bf16", "f32", 0, 40009, 127),
    ("bf16", None, "e4m3", 32, 20011, 131), ("bf16", "bf16", "e4m3", 128, 3001, 301), ("f32", None, "e4m3", 64, 20011, 33), ("bf16", "f32", "e4m3", 0, 701, 5003),
    ("bf16", None, "bf16", 0, 80003, 32), ("bf16", "f32", "e4m3", 32, 40009, 64), ("f32", "f32", "e4m3", 128, 20011, 136), ("bf16", "bf16", "f32", 0, 9001, 512)])
def test_norm_of_many_rows(x, res, out, block, rows, width):
    """Narrow and odd rows, several turns of every CTA."""
    xs = (ref.rnd(1, rows, width) * 2).to(DT[x]).cuda()
    r = None if res is None else (ref.rnd(2, rows, width) * 5).to(DT[res]).cuda()
    check_norm(xs, (1 + 0.1 * ref.rnd(3, width)).cuda(), r, out, block)


@pytest.mark.parametrize("width", [1, 5, 17, 40, 200])
@pytest.mark.parametrize("x,res", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_norm_at_every_start(x, res, width):
    """x, residual and sum each at an offset of its own, as views of larger buffers that keep what is around them."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    gain = (1 + 0.1 * ref.rnd(3, width)).cuda()
    for start in range(9):
        xb, rb = (ref.rnd(1, 4 * width + 9) * 2).to(DT[x]).cuda(), (ref.rnd(2, 4 * width + 9) * 5).to(DT[res]).cuda()
        xs = xb[start:start + 3 * width].view(3, width)
        rs = rb[(start * 5) % 9:][:3 * width].view(3, width)
        check_norm(xs, gain, rs, "bf16")
        want_y, want, _ = rms_norm(xs, gain, residual=rs)
        before = rb.clone()
        y, s, _ = rms_norm(xs, gain, residual=rs, sum_out=rs)   # in place
        assert s is rs and torch.equal(rs, want) and torch.equal(y, want_y)
        rs.copy_(before[(start * 5) % 9:][:3 * width].view(3, width))
        assert torch.equal(rb, before)


@pytest.mark.parametrize("out", ["f32", "e4m3"])
def test_norm_of_heads_in_strides(out):
    """Heads of a fused projection (rows and heads at strides of their own), written in strides, odd starts."""
    buf = ref.rnd(1, 6, 5 * 64 + 3).cuda()
    q = torch.as_strided(buf, (6, 3, 64), (5 * 64 + 3, 64, 1), 1)
    gain = (1 + 0.1 * ref.rnd(2, 64)).cuda()
    y = torch.zeros(6, 4, 65, dtype=DT[out], device="cuda")
    view = y[:, :3, :64]
    check_norm(q, gain, None, out, 32 if out == "e4m3" else 0, into=view)
    assert (y[:, 3].float() == 0).all() and (y[:, :, 64].float() == 0).all()
    assert torch.equal(buf, ref.rnd(1, 6, 5 * 64 + 3).cuda())
    check_norm(q.contiguous().view(2, 3, 3, 64), gain, None, out)


@pytest.mark.parametrize("width", [64, 1000, 20000])
def test_norm_in_place(width):
    from kv_cached_qwen3_gb300.norm import rms_norm
    x, r = ref.rnd(1, 5, width).cuda(), ref.rnd(2, 5, width).cuda()
    gain = (1 + 0.1 * ref.rnd(3, width)).cuda()
    y, s, _ = rms_norm(x, gain, residual=r)
    x2, r2 = x.clone(), r.clone()
    y2, s2, _ = rms_norm(x2, gain, residual=r2, out=x2, sum_out=r2)
    assert y2.data_ptr() == x2.data_ptr() and torch.equal(x2, y) and torch.equal(r2, s)
    x3 = x.clone()
    y3, s3, _ = rms_norm(x3, gain, residual=r, sum_out=x3)
    assert torch.equal(x3, s) and torch.equal(y3, y)


def test_norm_of_unusual_values():
    from kv_cached_qwen3_gb300.norm import rms_norm
    gain = torch.ones(64).cuda()
    x = ref.rnd(1, 6, 64).cuda()
    x[0] = 0
    x[1, 3] = math.nan
    x[2, 5] = math.inf
    x[3] *= 1e-20
    x[4] *= 1e15
    y = rms_norm(x, gain)[0].cpu()
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 5].isnan() and (y[2, :5] == 0).all()
    want, _ = ref.rms_norm(x[3:].cpu(), gain.cpu(), 1e-6)
    assert_within(y[3:], want, want.abs() * 40 * STEP)
    c, _, scales = rms_norm(x, gain, out_dtype=torch.float8_e4m3fn, block=32)
    v = c.float().cpu() * ref.by_block(scales.cpu(), 32, 64)
    assert (v[0] == 0).all() and v[1].isnan().all() and v[2, :32].isnan().all() and (v[2, 32:] == 0).all() and v[3:].isfinite().all()
    z = rms_norm(x[:1], gain, eps=0.0)[0]
    assert z.isnan().all()          # 0 / 0
    assert rms_norm(x[:0], gain)[0].shape == (0, 64)


def test_norm_refusals():
    from kv_cached_qwen3_gb300.norm import rms_norm
    x, g = torch.zeros(4, 64).cuda(), torch.ones(64).cuda()
    for args, kw in (((x.half(), g), {}), ((x.cpu(), g), {}), ((x.t(), g), {}), ((x, g[:32]), {}), ((x, g.bfloat16()), {}), ((x[0], g), {}),
                     ((x, g), dict(residual=x[:2])), ((x, g), dict(residual=x.half())), ((x, g), dict(out_dtype=torch.float16)),
                     ((x, g), dict(block=48)), ((x, g), dict(sum_out=x)), ((x, g), dict(out=x[:2])), ((x, g), dict(residual=x, sum_out=x.bfloat16())),
                     ((x.view(2, 2, 2, 32)[:, :, :, :16], g[:16]), {})):
        with pytest.raises(ValueError):
            rms_norm(*args, **kw)


# ------------------------------------------------------------------ rotary

SCALED = [None, dict(type="linear", factor=4.0), dict(type="ntk", factor=2.5), dict(type="smooth", factor=8.0, original=8192, low=1.0, high=4.0),
          dict(type="yarn", factor=4.0, original=4096, beta_fast=32.0, beta_slow=1.0), dict(type="yarn", factor=4.0, original=4096, beta_fast=16.0, beta_slow=2.0, amplitude=0.75)]


def turn_bound(size, dtype):
    """cos and sin within 2^-22 (a place in the turn within 2^-32, an eighth of a turn rounded to f32, 2 units of f32), two
    products and a sum rounded, and the result's own rounding."""
    return size * (2.0 ** -21 + ref.half_step(dtype) * (dtype is not torch.float32))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hd,rd", [(2, 2), (6, 4), (64, 64), (128, 128), (128, 64), (80, 40), (96, 30), (256, 256), (66, 66)])
def test_rotate(dt, interleaved, hd, rd):
    from kv_cached_qwen3_gb300.rotary import Rotary
    for i, scaling in enumerate(SCALED):
        if scaling and scaling["type"] == "ntk" and rd < 4:
            continue
        rows, theta = (1, 5, 67)[i % 3], (1e4, 1e6)[i % 2]
        q, k = ref.rnd(i, rows, 3, hd).to(DT[dt]), ref.rnd(50 + i, rows, 2, hd).to(DT[dt])
        pos = torch.randint(0, 200000, (rows,), generator=torch.Generator().manual_seed(i), dtype=torch.int32)
        pos[0] = 0
        r = Rotary(hd, rotary_dim=rd, theta=theta, interleaved=interleaved, scaling=scaling)
        got = r.rotate(q.cuda(), k.cuda(), pos.cuda())
        for t, y in zip((q, k), got):
            want, size = ref.rotate(t, pos, rd, theta, scaling, interleaved)
            assert_within(y, want, turn_bound(size, y.dtype))
            assert torch.equal(y[..., rd:].cpu(), t[..., rd:])
            if not (scaling and scaling["type"] == "yarn"):
                assert torch.equal(y[0].cpu(), t[0])                      # position 0


def test_rotate_far_and_negative_positions():
    from kv_cached_qwen3_gb300.rotary import Rotary
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 1, 10 ** 9, -12345], dtype=torch.int32)
    x = ref.rnd(1, 6, 2, 64)
    r = Rotary(64, theta=1e4)
    y = r.rotate(x.cuda(), None, pos.cuda())
    assert y[1] is None
    want, size = ref.rotate(x, pos, 64, 1e4, None, False)
    # 2^31 positions times 2^-54 turn of the table's own f64 frequencies, and as much of the reference's
    assert_within(y[0], want, turn_bound(size, torch.float32) + size * 2 ** 31 * 2.0 ** -51)
    back = r.rotate(y[0][2:], None, -pos[2:].cuda())[0]
    assert_within(back, x[2:], 2 * turn_bound(size[2:], torch.float32) + size[2:] * 2.0 ** -21)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_in_strides_and_in_place(dt, interleaved):
    """q and k as parts of a fused projection of several streams, at odd places; in place, and into a cache's layout."""
    from kv_cached_qwen3_gb300.rotary import Rotary
    B, T, D = 3, 7, 32
    for off, pad in ((0, 0), (1, 3), (2, 2), (4, 4)):
        buf = ref.rnd(1, B * (T * (9 * D + pad) + 5) + off).to(DT[dt]).cuda()
        stride = (T * (9 * D + pad) + 5, 9 * D + pad, D, 1)
        q = torch.as_strided(buf, (B, T, 5, D), stride, off)
        k = torch.as_strided(buf, (B, T, 2, D), stride, off + 5 * D)
        v = torch.as_strided(buf, (B, T, 2, D), stride, off + 7 * D)
        pos = torch.randint(0, 5000, (B, T), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
        r = Rotary(D, rotary_dim=24, interleaved=interleaved)
        v0 = v.clone()
        want = [ref.rotate(t.cpu(), pos, 24, 1e6, None, interleaved) for t in (q, k)]
        q2, k2 = r.rotate(q, k, pos.cuda())
        into = torch.zeros(2, B, T, D, dtype=DT[dt], device="cuda").permute(1, 2, 0, 3)
        _, k3 = r.rotate(q, k, pos.cuda(), out=(torch.empty_like(q2), into))
        assert torch.equal(k3, k2)
        r.rotate(q, k, pos.cuda(), out=(q, k))
        for y, z, (w, size) in ((q2, q, want[0]), (k2, k, want[1])):
            assert_within(y, w, turn_bound(size, y.dtype))
            assert torch.equal(y, z)
        assert torch.equal(v, v0)


def test_rotate_no_rows_and_no_heads():
    from kv_cached_qwen3_gb300.rotary import Rotary
    r = Rotary(64)
    pos = torch.zeros(4, dtype=torch.int32).cuda()
    q, k = r.rotate(torch.zeros(0, 2, 64).cuda(), None, pos[:0])
    assert q.shape == (0, 2, 64) and k is None
    x = ref.rnd(1, 4, 3, 64).cuda()
    q, k = r.rotate(x[:, :0], x, pos)
    assert q.shape == (4, 0, 64) and torch.equal(k, x)
    q, k = r.rotate(x, x[:, :0], pos)
    assert torch.equal(q, x) and k.shape == (4, 0, 64)


def test_rotate_refusals():
    from kv_cached_qwen3_gb300.rotary import Rotary
    for kw in (dict(head_dim=0), dict(head_dim=513), dict(head_dim=64, rotary_dim=63), dict(head_dim=64, rotary_dim=66), dict(head_dim=64, scaling=dict(type="x")),
               dict(head_dim=64, scaling=dict(type="linear")), dict(head_dim=64, scaling=dict(type="linear", factor=2.0, low=1.0))):
        with pytest.raises(ValueError):
            Rotary(**kw)
    with pytest.raises(RuntimeError):
        Rotary(64, theta=0.5)
    r = Rotary(64)
    x, pos = torch.zeros(4, 2, 64).cuda(), torch.zeros(4, dtype=torch.int32).cuda()
    for args, kw in (((x.half(), None, pos), {}), ((x, x.bfloat16(), pos), {}), ((x[0], None, pos), {}), ((x, None, pos.long()), {}), ((x, None, pos[:2]), {}),
                     ((x.cpu(), None, pos), {}), ((x[..., :32], None, pos), {}), ((x, x[:2], pos), {}), ((x, None, pos.cpu()), {}), ((x, None, pos), dict(out=(x[:2],)))):
        with pytest.raises(ValueError):
            r.rotate(*args, **kw)


# ------------------------------------------------------------------ 4-bit products

def check_product(rows, n, k, group, x, out, zeros, res, gated, seed=0, block=128, xv=None):
    """A product c x of a code and an input is exact, or has 22 bits of x. The tensor cores add sixteen at a time to a group's
    sum, cut off after 2^-23 of its largest value, which is at most sum |c - z| |x| <= 15 sum |x|, and seventeen numbers may
    be cut off (45 allows for three); totals of groups, of warps and of parts follow, f32 roundings of numbers up to that."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    m = [ref.w4_matrix(seed + i, n, k, group, zeros) for i in range(2 if gated else 1)]
    W = W4Matrix.pack(*[None if t is None else t.cuda() for t in m[0]], k=k, group=group,
                      gated_with=[None if t is None else t.cuda() for t in m[1]] if gated else None)
    xv = ref.rnd(seed + 5, rows, k) if xv is None else xv
    xs, xd = None, xv.to(DT[x]) if x != "e4m3" else None
    if x == "e4m3":
        c, _, s = rms_norm(xv.cuda(), torch.ones(k).cuda(), out_dtype=torch.float8_e4m3fn, block=block)
        xd, xs = c, s
        x64 = c.float().cpu().double() * ref.by_block(s.cpu().double(), block, k)
    else:
        x64 = xd.double()
    r = (10 * ref.rnd(seed + 6, rows, n)).to(DT[out]) if res else None
    y = W.matmul(xd.cuda(), x_scales=xs, residual=None if r is None else r.cuda(), out_dtype=DT[out])
    ws = [ref.w4_values(*t, k, group) for t in m]
    prod = [x64 @ w.T for w, _ in ws]
    size = [45 * (x64.abs() @ d.abs().T) for _, d in ws]
    roundings = group / 16 + -(-k // group) / 4 + 16
    err = [s * roundings * 2.0 ** -23 for s in size]
    if gated:
        g, u = prod
        want = g * torch.sigmoid(g) * u
        # |silu'| <= 1.1
        err = 1.1 * err[0] * (u.abs() + err[1]) + (g.abs() + err[0]) * err[1] + want.abs() * 2.0 ** -20
    else:
        want, err = prod[0], err[0]
    if r is not None:
        want = want + r.double()
    assert y.shape == (rows, n) and y.dtype is DT[out]
    assert_within(y, want, err + want.abs() * (STEP * 2 + ref.half_step(y.dtype) * (out != "f32") * (1 + STEP)))
    # and as a whole no worse than f32 sums: a root of the terms' roundings, not their sum
    if out == "f32" and k >= 64 and not gated and r is None:
        assert float((y.double().cpu() - want).norm() / want.norm()) <= 1e-6
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x,out,zeros,res,gated", [("f32", "f32", False, False, False), ("bf16", "f32", True, False, False), ("e4m3", "f32", False, True, False),
                                                   ("bf16", "bf16", False, True, False), ("f32", "bf16", True, False, True), ("bf16", "f32", False, False, True)])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 1), (1, 16, 128), (2, 7, 33), (3, 33, 2), (4, 17, 129), (5, 100, 300), (8, 48, 1000), (9, 31, 65), (17, 40, 127), (33, 64, 256), (65, 24, 383),
                                      (130, 9, 64)])
def test_product(group, x, out, zeros, res, gated, rows, n, k):
    check_product(rows, n, k, group, x, out, zeros, res, gated, seed=rows + n)


@pytest.mark.parametrize("rows,n,k,group,x", [(1, 500, 8192, 32, "f32"), (1, 300, 5000, 128, "e4m3"), (16, 700, 2100, 64, "bf16"), (64, 200, 4097, 128, "bf16"), (3, 5003, 1500, 32, "f32"),
                                              (1, 20000, 512, 64, "bf16"), (40, 3000, 640, 32, "e4m3"), (2, 64, 20000, 128, "f32")])
def test_larger_products(rows, n, k, group, x):
    check_product(rows, n, k, group, x, "f32", rows % 2 == 0, False, False, seed=3)


@pytest.mark.parametrize("block", [0, 32, 64, 128])
def test_product_of_rows_in_8_bits(block):
    for k in (30, 64, 130, 1000):
        check_product(3, 50, k, 64, "e4m3", "f32", False, False, False, block=block)


def test_product_in_strides():
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    n, k = 37, 75
    m = ref.w4_matrix(1, n, k, 32, False)
    W = W4Matrix.pack(m[0].cuda(), m[1].cuda(), k=k, group=32)
    for dt in (torch.float32, torch.bfloat16):
        x = ref.rnd(2, 5, k).to(dt).cuda()
        y = W.matmul(x)
        buf = torch.zeros(5, k + 3, dtype=dt, device="cuda")
        buf[:, 1:1 + k] = x
        out = torch.full((5, n + 5), 7.0, dtype=dt, device="cuda")
        W.matmul(buf[:, 1:1 + k], out=out[:, 2:2 + n])
        assert torch.equal(out[:, 2:2 + n], y) and (out[:, :2] == 7).all() and (out[:, 2 + n:] == 7).all()
        r = ref.rnd(3, 5, n).to(dt).cuda()
        z = W.matmul(x, residual=r)
        assert W.matmul(x, residual=r, out=r) is r and torch.equal(r, z)
        assert torch.equal(W.matmul(x[3:4]), y[3:4])           # a row's result does not depend on the others
        assert W.matmul(x[:0]).shape == (0, n)


def test_product_of_unusual_rows():
    """Rows of zeros, of very large and very small values, with a NaN or an infinity, and of values far apart."""
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    n, k = 20, 200
    m = ref.w4_matrix(1, n, k, 64, True)
    W = W4Matrix.pack(*[t.cuda() for t in m], k=k, group=64)
    w, d = ref.w4_values(*m, k, 64)
    for dt in (torch.float32, torch.bfloat16):
        x = ref.rnd(2, 9, k)
        x[0] = 0
        x[1] *= 1e37
        x[2] *= 1e-30
        x[3, 7] = math.nan
        x[4, 199] = -math.inf
        x[5, ::2] *= 1e-7
        x[6] *= 1e-41
        x[7, 1:] = 0
        x = x.to(dt)
        y = W.matmul(x.cuda(), out_dtype=torch.float32).cpu()
        assert (y[0] == 0).all() and y[3].isnan().all() and y[4].isnan().all()
        for r in (1, 2, 5, 6, 7, 8):
            want = x[r].double() @ w.T
            size = 45 * (x[r].double().abs() @ d.abs().T)
            assert_within(y[r], want, size * 30 * 2.0 ** -23 + 45 * k * d.abs().amax() * 1e-45 * (2.0 ** 14 if r == 6 else 1) + 1e-38)


def test_product_of_nan_scales():
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    m = ref.w4_matrix(1, 18, 130, 64, False)
    m[1][3, 1] = math.nan
    m[1][17, 2] = math.inf
    y = W4Matrix.pack(m[0].cuda(), m[1].cuda(), k=130, group=64).matmul(ref.rnd(1, 2, 130).cuda()).cpu()
    bad = ~y.isfinite()
    assert bad[:, [3, 17]].all() and int(bad.sum()) == 4


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 31), (5, 64), (4, 129), (7, 1000)])
def test_quantize(dt, group, n, k):
    import kv4_ref
    import numpy as np
    from kv_cached_qwen3_gb300.w4 import W4Matrix, quantize
    w = ref.rnd(n + k, n, k)
    w[0, : group // 2] *= 1e-38 if n > 1 else 1
    if n > 3:
        w[1] = torch.randint(-8, 9, (k,), generator=torch.Generator().manual_seed(1)) / 8.0     # borders, ties of both signs
        w[2] = 0
        w[3, :2] = torch.tensor([1e6, -1e30])
    w = w.to(DT[dt])
    buf = torch.zeros(n, k + 3, dtype=DT[dt]).cuda()
    buf[:, :k] = w
    codes, scales = quantize(buf[:, :k], group)
    pad = torch.zeros(n, -k % group, dtype=F64)
    full = torch.cat([w.double(), pad], 1).numpy().reshape(-1, group)
    at = np.argmax(np.abs(full), -1)[:, None]
    m = np.clip(np.take_along_axis(full, at, 1), -524032.0, 524032.0)
    c = np.zeros(full.shape, np.int64)
    for j in range(1, 16):
        c += np.where(m > 0, -16.0 * full >= (2 * j - 17) * m, -16.0 * full <= (2 * j - 17) * m)
    c = np.where(m == 0, 8, c).reshape(n, -1)[:, :k]
    got = torch.stack([codes & 15, codes >> 4], -1).flatten(1)[:, :k].cpu().numpy()
    np.testing.assert_array_equal(got, c)
    np.testing.assert_array_equal(scales.cpu().numpy().reshape(-1).view(np.uint16), (m[:, 0] / -8.0).astype(np.float32).astype(np.float16).view(np.uint16))
    if group == 32 and k % 32 == 0:                                # the cache's own blocks
        want = kv4_ref.q4_quantize(w.double().numpy())
        np.testing.assert_array_equal(got, want[0])
    W = W4Matrix.quantize(buf[:, :k], group)
    x = ref.rnd(9, 2, k)
    vals, d = ref.w4_values(codes.cpu(), scales.cpu(), None, k, group)
    assert_within(W.matmul(x.cuda()), x.double() @ vals.T, 45 * (x.double().abs() @ d.abs().T) * 64 * 2.0 ** -23 + 1e-38)


def test_quantize_bad_groups():
    from kv_cached_qwen3_gb300.w4 import quantize
    w = ref.rnd(1, 4, 96)
    w[1, 40], w[2, 5], w[3, 90] = math.nan, math.inf, -math.inf
    codes, scales = quantize(w.cuda(), 32)
    bad = scales.isnan().cpu()
    assert bad.nonzero().tolist() == [[1, 1], [2, 0], [3, 2]]
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(1).cpu()
    assert (n[1, 32:64] == 8).all() and (n[2, :32] == 8).all() and (n[3, 64:] == 8).all()


def test_product_refusals():
    from kv_cached_qwen3_gb300.w4 import W4Matrix, quantize
    c, s = (t.cuda() for t in ref.w4_matrix(1, 16, 64, 32, False)[:2])
    for args, kw in (((c, s), dict(k=64, group=48)), ((c, s), dict(k=62, group=32)), ((c.int(), s), dict(k=64, group=32)), ((c, s.float()), dict(k=64, group=32)),
                     ((c, s[:, :1]), dict(k=64, group=32)), ((c, s, s), dict(k=64, group=32)), ((c.cpu(), s.cpu()), dict(k=64, group=32)),
                     ((c, s), dict(k=64, group=32, gated_with=(c[:8], s))), ((c, s), dict(k=64, group=32, gated_with=(c, s, c[:, :2].contiguous())))):
        with pytest.raises(ValueError):
            W4Matrix.pack(*args, **kw)
    for w, g in ((torch.zeros(4, 64).cuda(), 16), (torch.zeros(4, 64), 32), (torch.zeros(4, 64).cuda().half(), 32), (torch.zeros(64, 4).cuda().t(), 32), (torch.zeros(0, 64).cuda(), 32)):
        with pytest.raises(ValueError):
            quantize(w, g)
    W = W4Matrix.pack(c, s, k=64, group=32)
    x = torch.zeros(3, 64).cuda()
    x8 = x.to(torch.float8_e4m3fn)
    for args, kw in (((x.half(),), {}), ((x[:, :32],), {}), ((x.cpu(),), {}), ((x8,), {}), ((x8, x[:, :3].contiguous()), {}), ((x8, x[:2, :2].contiguous()), {}), ((x8, x[:, :2].bfloat16().contiguous()), {}),
                     ((x, x[:, :2].contiguous()), {}), ((x,), dict(out_dtype=torch.float16)), ((x,), dict(out=x)), ((x,), dict(residual=x)), ((x,), dict(residual=x[:, :16].bfloat16()))):
        with pytest.raises(ValueError):
            W.matmul(*args, **kw)
