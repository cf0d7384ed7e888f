"""GPU: tensors whose last dimension has one element, which then has no stride that counts."""
import pytest

import layer_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def odd(t):
    """t [..., 1] with another stride in its last dimension."""
    v = torch.as_strided(t.contiguous().clone(), t.shape, t.contiguous().stride()[:-1] + (7,))
    assert v.stride(-1) == 7 and torch.equal(v, t)
    return v


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_norm_of_single_values(dt):
    from kv_cached_qwen3_gb300.norm import rms_norm
    gain = torch.full((1,), 1.5).cuda()
    for shape in ((5, 1), (4, 3, 1), (2, 2, 3, 1)):
        x, r = ref.rnd(1, *shape).to(dt).cuda(), ref.rnd(2, *shape).to(dt).cuda()
        want = rms_norm(x, gain, residual=r)
        got = rms_norm(odd(x), gain, residual=odd(r), out=odd(torch.zeros_like(x)), sum_out=odd(torch.zeros_like(r)))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(rms_norm(x.flatten()[None].t(), gain)[0].flatten(), rms_norm(x, gain)[0].flatten())


def test_products_of_single_values():
    from kv_cached_qwen3_gb300.w4 import W4Matrix, quantize
    w = ref.rnd(1, 5, 1).cuda()
    codes, scales = quantize(odd(w), 32)
    assert torch.equal(codes, quantize(w, 32)[0]) and torch.equal(scales, quantize(w, 32)[1])
    x = ref.rnd(2, 4, 1).cuda()
    one = W4Matrix.quantize(odd(w), 32)
    assert torch.equal(one.matmul(odd(x)), one.matmul(x))
    v, y, r = ref.rnd(3, 1, 40).cuda(), ref.rnd(4, 4, 40).cuda(), ref.rnd(5, 4, 1).cuda()
    row = W4Matrix.quantize(v, 32)
    out = odd(torch.zeros(4, 1).cuda())
    assert row.matmul(y, residual=odd(r), out=out) is out and torch.equal(out, row.matmul(y, residual=r))


def test_drafts_over_one_token():
    from kv_cached_qwen3_gb300.draft import draft_verify
    t, d = ref.rnd(1, 3, 3, 1).cuda(), ref.rnd(2, 3, 2, 1).cuda()
    tokens, u = torch.zeros(3, 2, dtype=torch.int32).cuda(), ref.uni(3, 3, 3).cuda()
    for a, b in zip(draft_verify(odd(t), tokens, u, draft_logits=odd(d)), draft_verify(t, tokens, u, draft_logits=d)):
        assert torch.equal(a, b)


def test_rows_that_all_read_one_place():
    """Inputs that rows share, and results that they would: the first are taken, the second refused."""
    from kv_cached_qwen3_gb300.norm import rms_norm
    from kv_cached_qwen3_gb300.rotary import Rotary
    from kv_cached_qwen3_gb300.talker import TalkerError
    for width in (64, 47):
        x, r, gain = ref.rnd(1, 5, width).cuda(), ref.rnd(2, 1, width).cuda(), torch.ones(width).cuda()
        y, s, _ = rms_norm(x, gain, residual=r.expand(5, width))
        y2, s2, _ = rms_norm(x, gain, residual=r.expand(5, width).contiguous())
        assert torch.equal(y, y2) and torch.equal(s, s2)
        with pytest.raises(TalkerError):
            rms_norm(x, gain, residual=r.expand(5, width), sum_out=r.expand(5, width))
        with pytest.raises(TalkerError):
            rms_norm(x, gain, out=torch.zeros(1, width).cuda().expand(5, width))
        h = ref.rnd(3, 4, 1, width).cuda()
        z = rms_norm(h.expand(4, 3, width), gain)[0]
        assert torch.equal(z, rms_norm(h, gain)[0].expand(4, 3, width))
        with pytest.raises(TalkerError):
            rms_norm(h.expand(4, 3, width), gain, out=h.expand(4, 3, width))
    rope, pos = Rotary(64), torch.arange(4, dtype=torch.int32).cuda()
    q = ref.rnd(4, 4, 1, 64).cuda()
    turned = rope.rotate(q, None, pos)[0]
    assert torch.equal(rope.rotate(q.expand(4, 3, 64), None, pos)[0], turned.expand(4, 3, 64))
    before = q.clone()
    with pytest.raises(TalkerError):
        rope.rotate(q.expand(4, 3, 64), None, pos, out=(q.expand(4, 3, 64),))
    assert torch.equal(q, before)
    assert torch.equal(rope.rotate(q, None, pos, out=(q,))[0], turned)
