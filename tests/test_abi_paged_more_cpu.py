"""More of the paged calls without a GPU: overlapping arrays, tensors of another
device."""
import pytest

from test_abi_paged_cpu import INVALID, P, _append, _chunk, _dims


def test_append_refuses_queries_that_overlap_in_part():
    size = 4 * 8 * 32 * 2                                   # four tokens, eight heads of 32 bf16 channels
    for off in (16, size - 16):
        assert _append(q=P, qo=P + off) == INVALID
        assert _append(q=P + off, qo=P) == INVALID
    none = dict(B=0)                                        # no sequences: the arguments are sound and nothing runs
    assert _append(q=P, qo=P + size, **none) == 0 and _append(q=P + size, qo=P, **none) == 0
    assert _append(q=P, qo=P, **none) == 0
    assert _append(q=P, qo=P + 16, chunk=_chunk(N=0), **none) == 0
    f32 = _dims(dtype="f32")
    assert _append(d=f32, q=P, qo=P + 2 * size - 16) == INVALID
    assert _append(d=f32, q=P, qo=P + 2 * size, **none) == 0


class _On:
    """Stands in for a tensor on a device."""

    def __init__(self, dev, ptr=P):
        self.dev, self.ptr = dev, ptr

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return self.ptr


def _calls(mtla):
    """Every binding: its number of tensors, those of its structs among them, and a call of B = 0 sequences."""
    d = _dims()

    def chunk(x):
        return mtla.chunk(0, x[0], x[1], x[2])

    def append(x):
        x = list(x)
        c, m = chunk(x), mtla.merge_args(*x[3:8], 4)
        pages = mtla.paged_cache(x[8], 10, 16, 288, x[9], 2)
        mtla.mtla_paged_append(d, 0, c, m, 1e4, x[10], x[11], pages, x[12], x[13], x[14], x[15], x[16], x[17], 0, x[18], stream=0)

    def attn(x):
        pages = mtla.paged_cache(x[3], 10, 16, 288, x[4], 2)
        mtla.mtla_paged_attn(d, 0, chunk(x), x[5], x[6], x[7], pages, x[8], mtla.MTLA_BF16, x[9], x[10], 0, x[11], stream=0)

    def verify(x):
        mtla.mtla_verify_drafts(0, 0, 10, x[0], 10, x[1], 10, *x[2:9], stream=0)

    return (append, 19), (attn, 12), (verify, 9)


@pytest.mark.parametrize("which", [0, 1, 2], ids=["append", "attn", "verify"])
def test_tensors_of_another_device_are_refused(monkeypatch, which):
    torch = pytest.importorskip("torch")
    import temporally_compressed_latent_b200 as mtla
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    call, n = _calls(mtla)[which]
    call([_On(1)] * n)                                  # all where they belong: nothing to do, nothing refused
    for k in range(n):
        for other, name in ((_On(0), "cuda:0"), (torch.zeros(8, dtype=torch.uint8), "the host")):
            x = [_On(1) for _ in range(n)]
            x[k] = other
            with pytest.raises(ValueError, match=f"on {name}, the current device is cuda:1"):
                call(x)
            x = [P] * n                                 # addresses say nothing about their device
            x[k] = other
            with pytest.raises(ValueError, match=f"on {name}, the current device is cuda:1"):
                call(x)
    call([P] * n)
