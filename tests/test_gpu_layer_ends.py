"""GPU: the operators around a layer's attention at the ends of what they take: most sequences and rows, broadcast and odd
places, unusual values in odd rows, threads at once."""
import math
import threading

import pytest

import layer_ref as ref
from test_gpu_draft import check as check_draft, inputs as draft_inputs
from test_gpu_layer import STEP, assert_within, check_norm, check_product

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("width", [13, 65, 1001, 40001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_odd_norm_in_place(width, dt):
    """y over x and s over the residual, rows that arrive while others are written."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    rows = 20011 if width < 100 else 700 if width < 2000 else 3
    t = torch.float32 if dt == "f32" else torch.bfloat16
    x, r = ref.rnd(1, rows, width).to(t).cuda(), ref.rnd(2, rows, width).to(t).cuda()
    gain = (1 + 0.1 * ref.rnd(3, width)).cuda()
    y, s, _ = rms_norm(x, gain, residual=r)
    x2, r2 = x.clone(), r.clone()
    rms_norm(x2, gain, residual=r2, out=x2, sum_out=r2)
    assert torch.equal(x2, y) and torch.equal(r2, s)
    x3, r3 = x.clone(), r.clone()
    rms_norm(x3, gain, residual=r3, out=r3, sum_out=x3)
    assert torch.equal(r3, y) and torch.equal(x3, s)


@pytest.mark.parametrize("width", [64, 67, 1000, 4099])
def test_norm_of_one_row_for_all(width):
    """A residual and an x at a stride of zero."""
    x, r = (ref.rnd(1, 300, width) * 2).cuda(), (ref.rnd(2, 1, width) * 5).cuda()
    gain = (1 + 0.1 * ref.rnd(3, width)).cuda()
    check_norm(x, gain, r.expand(300, width), "bf16")
    check_norm(r.expand(300, width), gain, x, "e4m3", block=64)


@pytest.mark.parametrize("block", [0, 32, 64, 128])
def test_unusual_values_in_odd_rows(block):
    from kv_cached_qwen3_gb300.norm import rms_norm
    width = 257
    gain = torch.ones(width).cuda()
    x = ref.rnd(1, 6, width).cuda()
    x[0] = 0
    x[1, 256] = math.nan
    x[2, 5] = -math.inf
    x[3] *= 1e-20
    x[4] *= 1e15
    y = rms_norm(x, gain)[0].cpu()
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 5].isnan() and (y[2, :5] == 0).all()
    want, _ = ref.rms_norm(x[3:].cpu(), gain.cpu(), 1e-6)
    assert_within(y[3:], want, want.abs() * 40 * STEP)
    c, _, scales = rms_norm(x, gain, out_dtype=torch.float8_e4m3fn, block=block)
    v = c.float().cpu() * ref.by_block(scales.cpu(), block, width)
    of = block or width       # the infinity's block
    assert (v[0] == 0).all() and v[1].isnan().all() and v[2, :of].isnan().all() and (v[2, of:] == 0).all() and v[3:].isfinite().all()
    assert rms_norm(x[:1], gain, eps=0.0)[0].isnan().all()          # 0 / 0
    assert rms_norm(x[:0], gain)[0].shape == (0, width)


@pytest.mark.parametrize("S,K,V", [(130, 4, 300), (300, 2, 2048), (700, 1, 33), (64, 3, 9000), (33, 10, 4000)])
def test_many_sequences_verified(S, K, V):
    """Clusters of every size: they have fewer CTAs the more sequences there are."""
    from kv_cached_qwen3_gb300.draft import draft_verify
    t, d, tokens, u = draft_inputs(3, S, K, V, "bf16")
    check_draft(draft_verify, t, tokens, u, d)
    counts = torch.arange(S, dtype=torch.int32) % (K + 1)
    temps = 0.5 + ref.uni(9, S)
    temps[::4] = 0.0
    check_draft(draft_verify, t, tokens, u, None, counts, temps)


def test_most_sequences_verified():
    """65535 sequences, the most: 45 different ones over and over decide as they do by themselves."""
    from kv_cached_qwen3_gb300.draft import draft_verify
    t, d, tokens, u = (x.cuda() for x in draft_inputs(5, 45, 2, 70, "f32"))
    one = draft_verify(t, tokens, u, draft_logits=d)
    n = 65535 // 45 + 1
    rep = lambda x: x.repeat(n, *(1,) * (x.dim() - 1))[:65535].contiguous()
    many = draft_verify(rep(t), rep(tokens), rep(u), draft_logits=rep(d))
    assert torch.equal(many[0], rep(one[0])) and torch.equal(many[1], rep(one[1]))
    # (the f32 sums of taken drafts depend on how many parts a row is read in)
    assert ((many[2] - rep(one[2])).abs() <= (1 + rep(one[2]).abs() * 4) * 2.0 ** -19).all()


def test_logits_at_odd_places_of_many_sequences():
    """bf16 rows at every place in 16 bytes, with what is around them left out."""
    from kv_cached_qwen3_gb300.draft import draft_verify
    t, d, tokens, u = draft_inputs(7, 40, 3, 1001, "bf16")
    want = draft_verify(t.cuda(), tokens.cuda(), u.cuda(), draft_logits=d.cuda())
    for start in (1, 3, 6):
        tb = torch.full((40, 4, 1001 + 2 * start), 300.0, dtype=torch.bfloat16, device="cuda")
        db = torch.full((40, 3, 1001 + 2 * start), 300.0, dtype=torch.bfloat16, device="cuda")
        tv, dv = tb[:, :, start:start + 1001], db[:, :, start:start + 1001]
        tv.copy_(t)
        dv.copy_(d)
        got = draft_verify(tv, tokens.cuda(), u.cuda(), draft_logits=dv)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_most_rows_of_a_product(x):
    """65536 rows, in thousands of passes; one more is refused."""
    from kv_cached_qwen3_gb300.talker import TalkerError
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    check_product(65536, 24, 40, 32, x, "f32", True, False, False, seed=2)
    c, s, _ = ref.w4_matrix(2, 24, 40, 32, False)
    W = W4Matrix.pack(c.cuda(), s.cuda(), k=40, group=32)
    with pytest.raises(TalkerError):
        W.matmul(torch.zeros(65537, 40, device="cuda"))


def test_product_of_one_row_for_all():
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    c, s, z = ref.w4_matrix(2, 100, 300, 64, True)
    W = W4Matrix.pack(c.cuda(), s.cuda(), z.cuda(), k=300, group=64)
    x = ref.rnd(4, 1, 300).cuda()
    assert torch.equal(W.matmul(x.expand(9, 300)), W.matmul(x.repeat(9, 1)))


def test_rotation_of_one_row_for_all():
    """Heads and rows at a stride of zero are read, and written to places of their own."""
    from kv_cached_qwen3_gb300.rotary import Rotary
    r = Rotary(64)
    pos = torch.arange(7, dtype=torch.int32, device="cuda")
    q = ref.rnd(1, 1, 1, 64).cuda()
    got = r.rotate(q.expand(7, 5, 64), None, pos)[0]
    assert torch.equal(got, r.rotate(q.expand(7, 5, 64).contiguous(), None, pos)[0])


def test_threads_at_once():
    """Calls of several host threads, a stream each."""
    from kv_cached_qwen3_gb300.draft import draft_verify
    from kv_cached_qwen3_gb300.norm import rms_norm
    from kv_cached_qwen3_gb300.rotary import Rotary
    from kv_cached_qwen3_gb300.w4 import W4Matrix
    c, s, _ = ref.w4_matrix(1, 333, 200, 32, False)
    W, rope = W4Matrix.pack(c.cuda(), s.cuda(), k=200, group=32), Rotary(50, rotary_dim=20)
    t, d, tokens, u = (v.cuda() for v in draft_inputs(3, 4, 3, 700, "f32"))
    gain = torch.ones(200, device="cuda")

    def step(i):
        x = ref.rnd(i, 3 + i, 200).cuda()
        h, x, _ = rms_norm(x, gain, residual=x)
        q, _ = rope.rotate(x.view(3 + i, 4, 50), None, torch.arange(3 + i, dtype=torch.int32, device="cuda"))
        return [h, x, q, W.matmul(h), *draft_verify(t, tokens, u, draft_logits=d)]

    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    failed = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = step(i)
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        failed.append(i)
        except Exception as e:      # a thread's error is the test's
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed, failed
