"""A launch that CUDA refuses is reported by the call that made it, and by no other."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def P():
    import expert_ffn_gemv_b200 as P

    return P


class BrokenCapture:
    """A stream whose capture has been invalidated (by waiting for it): every launch on it is refused on the host,
    until the capture ends."""

    RELAXED = 2

    def __enter__(self):
        self.cuda = C.CDLL("libcuda.so.1")
        self.stream = torch.cuda.Stream()
        self.s = C.c_void_p(self.stream.cuda_stream)
        assert self.cuda.cuStreamBeginCapture_v2(self.s, self.RELAXED) == 0
        assert self.cuda.cuStreamSynchronize(self.s) != 0
        return self.stream

    def __exit__(self, *exc):
        graph = C.c_void_p()
        assert self.cuda.cuStreamEndCapture(self.s, C.byref(graph)) != 0 and not graph.value


def test_refused_launches(P):
    def randn(*s, dtype=F):
        return torch.randn(s, device="cuda").to(dtype)

    x, w = randn(3, 64), randn(64)
    many, wide = randn(2000, 1024), randn(1024)
    a, m = randn(12, 64, dtype=BF), randn(64, 64, dtype=BF)
    y, saved = P.ffn_forward(a, m, m, m, save=True)
    ad = P.Adapters(d_in=64, d_out=64, max_adapters=1, max_rank=8)
    ad.load(0, m[:8].contiguous(), m[:, :8].contiguous())
    xb, ids = randn(4, 64, dtype=BF), torch.zeros(4, dtype=torch.int32, device="cuda")
    rows, cols = m[:8].contiguous(), m[:, :8].contiguous()
    calls = {"norm_in": lambda: P.norm_in(x, w), "norm_in, many rows": lambda: P.norm_in(many, wide),
             "norm_out": lambda: P.norm_out(x, x, weight=w), "norm_in_backward": lambda: P.norm_in_backward(x, w, x)[0],
             "norm_in_backward, many rows": lambda: P.norm_in_backward(many, wide, many)[0],
             "norm_out_backward": lambda: P.norm_out_backward(x, x)[0], "ffn_forward, few": lambda: P.ffn_forward(a[:2], m, m, m),
             "ffn_forward": lambda: P.ffn_forward(a, m, m, m), "ffn_backward": lambda: P.ffn_backward(y, a, m, m, m, saved)[0],
             "apply": lambda: ad.apply(xb, xb, ids), "load": lambda: ad.load(0, rows, cols)}
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    for k, f in calls.items():
        with BrokenCapture() as s, torch.cuda.stream(s):
            with pytest.raises(P.MoeError) as e:
                f()
            assert e.value.status == P.MOE_ERR_CUDA, k
        for j, g in calls.items():  # whatever comes next is not blamed for it
            got = g()
            assert got is None or torch.equal(got, want[j]), (k, j)
    ad.close()
    assert P.block_check() == P.MOE_OK
