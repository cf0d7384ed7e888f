"""CPU: the strides that rms_norm hands to the library are its tensors' own for as long as the library may read them."""
import pytest

torch = pytest.importorskip("torch")


class Rows:
    """What rms_norm asks of a CUDA tensor [rows, heads, width], at an address of its own."""
    dtype, device = torch.float32, torch.device("cuda", 0)
    shape = torch.Size((2, 3, 8))

    def __init__(self, outer, inner):
        self.strides = (outer, inner, 1)

    def stride(self, dim=None):
        return self.strides if dim is None else self.strides[dim]

    def numel(self):
        return 48

    def data_ptr(self):
        return 4096


class Gain(Rows):
    def numel(self):
        return 8

    def is_contiguous(self):
        return True


def strides_read(monkeypatch, tensors, before):
    """What the library reads of a call's four tensors, `before` having run between the call's start and its read."""
    from kv_cached_qwen3_gb300 import norm
    read = []

    def launch(device, fn, what, *args):
        before()
        at = [args[i] for i in (2, 5, 12, 15)]
        held = [norm._RowStrides(7, 7) for _ in range(256)]     # takes the places that have become free
        read.extend((s.outer, s.inner) for s in map(norm._RowStrides.from_address, at))
        del held

    class Library:
        talker_rms_norm = None
    monkeypatch.setattr(norm, "launch", launch)
    monkeypatch.setattr(norm, "load_library", lambda: Library)
    x, res, s, y = tensors
    norm.rms_norm(x, Gain(8, 8), residual=res, sum_out=s, out=y)
    return read


def fill(first, count):
    from kv_cached_qwen3_gb300 import norm
    for i in range(count):
        norm._at(Rows(first + i, 8), 3)


@pytest.mark.parametrize("room", range(5))
def test_a_full_table_within_a_call(monkeypatch, room):
    """New strides while the table has room for 0 to 4 more, behind tensors whose strides it has."""
    from kv_cached_qwen3_gb300 import norm
    for known in range(4):
        norm._strides.clear()
        fill(1000, 4096 - room)
        strides = [(1000 + 5 * i, 8) if i <= known else (900000 + i, 16) for i in range(4)]
        assert strides_read(monkeypatch, [Rows(*s) for s in strides], lambda: None) == strides


def test_another_call_in_between(monkeypatch):
    """Calls of other threads, which run while this one is in the library."""
    from kv_cached_qwen3_gb300 import norm
    norm._strides.clear()
    strides = [(100 + i, 8 + i) for i in range(4)]
    assert strides_read(monkeypatch, [Rows(*s) for s in strides], lambda: fill(50000, 9000)) == strides
