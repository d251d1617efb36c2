"""What the binding lets through to the sparse and prefix calls: tensors of the
plan's sizes, type, layout and device.  The kernels read and write by the plan's
sizes, so anything else must be refused before the call.

The checks themselves run without a GPU on stand-ins for tensors; the public
calls' refusals are tested on the GPU, where nothing is launched."""
import pytest
import torch

from packed_varlen_non_gb300 import h3attn as H


class Fake:
    """A tensor's description, as if it lay on a device."""

    def __init__(self, shape, dtype=torch.bfloat16, strides=None, device=0):
        self.meta = torch.empty(shape, dtype=dtype, device="meta")
        if strides is not None:
            self.meta = self.meta.as_strided(shape, strides)
        self.shape, self.dtype, self.at = self.meta.shape, dtype, device
        self.device = f"cuda:{device}" if device >= 0 else "cpu"

    def get_device(self):
        return self.at

    def __getattr__(self, name):
        return getattr(self.meta, name)


SIZES = (10, 256, 0)  # ten tokens, two heads, device 0


def test_rows_lets_through_what_the_kernels_can_read():
    for t, stride in [(Fake((10, 256)), 256), (Fake((10, 2, 128)), 256), (Fake((12, 256)), 256),
                      (Fake((10, 2, 128), strides=(768, 128, 1)), 768),  # a slice of a fused buffer
                      (Fake((10, 768)), 768),                            # the buffer itself, its first columns
                      (Fake((10, 1, 256), strides=(256, 7, 1)), 256)]:   # a dimension of one has no stride
        assert H._rows((t, t), None, 10, SIZES) == stride
        assert H._rows((t,), stride, 10, SIZES) == stride
    assert H._rows((16, Fake((10, 256))), 256, 10, SIZES) == 256  # a raw pointer beside a tensor
    # one row has no stride: tensors that differ in it are the same to the kernels
    assert H._rows((Fake((1, 256), strides=(999, 1)), Fake((1, 2, 128))), None, 1, (1, 256, 0)) == 256


@pytest.mark.parametrize("bad", [
    Fake((9, 256)), Fake((10, 255)), Fake((10, 1, 128)), Fake((10, 256), dtype=torch.float16),
    Fake((10, 256), dtype=torch.float32), Fake((10, 256), dtype=torch.uint8), Fake((10, 256), strides=(1, 10)),
    Fake((10, 2, 128), strides=(512, 256, 1)), Fake((10, 2, 128), strides=(256, 128, 2)),
    Fake((10, 2, 128), strides=(128, 1280, 1)), Fake((2560,)), Fake((10, 2, 2, 64)), Fake((10, 256), device=-1),
    Fake((10, 256), device=1)])
def test_rows_refuses_other_tensors(bad):
    for tensors in ((bad,), (Fake((10, 256)), bad)):
        with pytest.raises(ValueError):
            H._rows(tensors, None, 10, SIZES)


def test_strides_have_to_agree():
    a, b = Fake((10, 256)), Fake((10, 256), strides=(512, 1))
    for tensors, given in (((a, b), None), ((a, a), 512), ((b,), 256), ((16, 16), None)):
        with pytest.raises(ValueError):
            H._rows(tensors, given, 10, SIZES)


def test_lse_is_fp32_and_whole():
    for t in (Fake((2, 10), dtype=torch.float32), Fake((20,), dtype=torch.float32), None, 16):
        H._check_lse(t, SIZES)
    for t in (Fake((2, 9), dtype=torch.float32), Fake((2, 11), dtype=torch.float32), Fake((2, 10)),
              Fake((2, 10), dtype=torch.float64), Fake((2, 10), dtype=torch.float32, strides=(11, 1)),
              Fake((2, 10), dtype=torch.float32, strides=(1, 2)), Fake((2, 10), dtype=torch.float32, device=-1),
              Fake((2, 10), dtype=torch.float32, device=1)):
        with pytest.raises(ValueError):
            H._check_lse(t, SIZES)


def test_the_stream_is_that_of_the_plans_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setitem(H._plan_device, 77, 3)
    assert H._plan_stream(77, None) == 1003 and H._plan_stream(78, None) == 1000
    assert H._plan_stream(77, 5) == 5 and H._plan_stream(77, 0) is None


@pytest.mark.gpu
def test_the_calls_refuse_them(lib):
    from tests import walk_cases as W
    from tests.gpu_cases import docs_1d
    with H.Plan(docs_1d([70, 30]), 2) as plan:
        p = plan.handle
        H.h3attn_plan_set_sparse(p, 256, 2)
        H.h3attn_plan_set_prefix(p, 40)
        q, k, v = (W.rows(100, 2, i) for i in range(3))
        kp, vp = (W.rows(40, 2, 3 + i) for i in range(2))
        idx = torch.zeros(2, 2, 2, dtype=torch.int32, device="cuda")
        cnt = torch.ones(2, 2, dtype=torch.int32, device="cuda")
        o, lse = W.outputs(100, 2)
        sel = dict(plan=p, q_hat=q, k_hat=k, keep=1, block_idx=idx, block_cnt=cnt)
        spa = dict(plan=p, q=q, k=k, v=v, block_idx=idx, block_cnt=cnt, o=o, softmax_scale=0.1, lse=lse)
        pre = dict(plan=p, q=q, k=k, v=v, k_prefix=kp, v_prefix=vp, o=o, softmax_scale=0.1, lse=lse)
        calls = ((H.h3attn_block_select, sel), (H.h3attn_forward_sparse, spa), (H.h3attn_forward_prefix, pre))
        for fn, kw in calls:
            fn(**kw)
            for name in ("q_hat", "k_hat", "q", "k", "v", "k_prefix", "v_prefix", "o"):
                if name not in kw:
                    continue
                t = kw[name]
                for bad in (t.float(), t.half(), t.view(torch.uint8), t[:-1], t[:, :1], t.transpose(0, 1), t.cpu(),
                            t.reshape(-1), t.transpose(1, 2).contiguous().transpose(1, 2)):
                    with pytest.raises(ValueError):
                        fn(**{**kw, name: bad})
            if "lse" in kw:
                for bad in (lse[:, :99], lse[:1], lse.half(), lse.double(), lse.t(), lse.cpu(),
                            torch.empty(2, 101, device="cuda")):
                    with pytest.raises(ValueError):
                        fn(**{**kw, "lse": bad})
                fn(**{**kw, "lse": None})
        torch.cuda.synchronize()
        H.h3attn_get_device_error(p)


@pytest.mark.gpu
def test_one_row_of_any_stride(lib):
    # a single token whose tensors come from buffers of different widths
    from oracle import walks
    from tests import walk_cases as W
    p, s = W.Prefix([1], 2, 1), W.Sparse([1], 2, 256, 1)
    q, k, v, kp, vp = (W.rows(1, 2, i) for i in range(5))
    wide = [W.strided(t, 256 + 8 * i) for i, t in enumerate((q, k, v, kp, vp))]
    wide = [t.as_strided((1, 256), (3, 1)) for t in wide]  # (a dimension of one may have any stride)
    o, lse = W.outputs(1, 2)
    H.h3attn_forward_prefix(p.plan.handle, *wide, W.flat(o), W.SCALE, lse)
    W.check(o, lse, q, [k, kp], walks.prefix_attention(*(W.f64(t) for t in (q, k, v, kp, vp)), p.cu, W.SCALE))
    H.h3attn_block_select(s.plan.handle, *wide[:2], 1, s.idx, s.cnt)
    assert s.idx.tolist() == [[[0]], [[0]]] and s.cnt.tolist() == [[1], [1]]
    H.h3attn_forward_sparse(s.plan.handle, *wide[:3], s.idx, s.cnt, W.flat(o), W.SCALE, lse)
    assert torch.equal(o, v)
