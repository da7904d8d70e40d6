"""Which GPU a call runs on (CPU: tensors without storage stand for those of two
GPUs, and a recorder for the library)."""
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import bf16_matrix_multiply_amd as bmm

pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer")


class Recorder:
    """Stands for the library: notes each launch with the device that is current and
    the stream it was given."""

    def __init__(self, state):
        self.state, self.launches = state, []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 1 << 12
            stream = getattr(args[-1], "value", args[-1])
            self.launches.append((name, self.state.device, stream))
            return 0
        return call


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs, the first of them current; the stream of GPU d is 1000 + d."""
    state = types.SimpleNamespace(device=0)

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state.device = state.device, self.index

        def __exit__(self, *exc):
            state.device = self.before

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=1000 + state.device))
    monkeypatch.setattr(bmm, "_current_device", lambda: state.device)
    monkeypatch.setattr(bmm, "_current_stream", lambda d: 1000 + d)
    recorder = Recorder(state)
    monkeypatch.setattr(bmm, "_lib", recorder)
    with FakeTensorMode(allow_non_fake_inputs=True):
        yield types.SimpleNamespace(state=state, launches=recorder.launches)


BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def empty(dtype, *shape):
    return lambda d: torch.empty(*shape, dtype=dtype, device=f"cuda:{d}")


def operand(rows, K):
    def make(d):
        codes, scales = bmm._mx4_shapes(1, rows, K)
        return bmm.Mx4Operand(empty(U8, *codes)(d), empty(U8, *scales)(d), rows, K)
    return make


X, H, W = empty(BF, 4, 32), empty(BF, 4, 24), empty(I32, 1, 3, 2, 8, 8)
A, B = empty(I32, 1, 1, 2, 16, 8), empty(I32, 1, 3, 2, 8, 8)
D = empty(torch.float32, 1, 1, 3, 16, 8)
XQ, WQ, BOX = operand(4, 64), operand(24, 64), empty(torch.float32, 8, 8)

CALLS = {  # the call, and its tensors: each a function of the GPU it is on
    "gated": (bmm.gated, [X, W, W]),
    "gated_out": (lambda x, g, u, o: bmm.gated(x, g, u, out=o), [X, W, W, H]),
    "gated_save": (lambda x, g, u: bmm.gated(x, g, u, save=True), [X, W, W]),
    "gated_keywords": (lambda x, g, u: bmm.gated(act="relu", X=x, Wg=g, Wu=u), [X, W, W]),
    "gated_backward": (bmm.gated_backward, [H, H, H, X, W, W]),
    "gated_backward_workspace": (lambda *t: bmm.gated_backward(*t[:6], workspace=t[6]),
                                 [H, H, H, X, W, W, empty(U8, 4096)]),
    "mx4_quantize": (bmm.mx4_quantize, [X]),
    "mx4_dequantize": (bmm.mx4_dequantize, [XQ]),
    "mx4_dequantize_out": (lambda q, o: bmm.mx4_dequantize(q, BF, o), [XQ, empty(BF, 4, 64)]),
    "mx4_mma": (bmm.mx4_mma, [XQ, WQ]),
    "mx4_mma_out": (lambda a, b, o: bmm.mx4_mma(a, b, BF, o), [XQ, WQ, H]),
    "mx4_gated": (bmm.mx4_gated, [XQ, WQ, WQ]),
    "mx4_gated_out": (lambda x, g, u, o: bmm.mx4_gated(x, g, u, out=o), [XQ, WQ, WQ, H]),
    "pack_operand": (lambda x: bmm.pack_operand(x, 8), [empty(BF, 8, 32)]),
    "pack_operand_out": (lambda x, o: bmm.pack_operand(x, 8, out=o),
                         [empty(BF, 24, 32), B]),
    "pack_operand_kmajor_out": (lambda x, o: bmm.pack_operand_kmajor(x, 8, out=o),
                                [empty(BF, 32, 24), B]),
    "mma_tile": (lambda a, b: bmm.mma_tile(a, b, dtype="bf16"), [A, B]),
    "mma_tile_c_out": (lambda a, b, c, o: bmm.mma_tile(a, b, c, dtype="bf16", out=o), [A, B, D, D]),
    "mma_tile_splitk": (lambda a, b: bmm.mma_tile_splitk(a, b, dtype="bf16", splits=1), [A, B]),
    "mma_tile_splitk_noalloc": (lambda a, b, o: bmm.mma_tile_splitk_noalloc(
        a, b, dtype="bf16", splits=1, out=o), [A, B, D]),
    "box_copy": (lambda s, o: bmm.box_copy(s, (4, 4), (0, 0), out=o), [BOX, empty(torch.float32, 1, 4, 4)]),
    "box_store": (lambda d, i: bmm.box_store(d, i, (4, 4), (0, 0)), [BOX, empty(torch.float32, 1, 4, 4)]),
    "box_reduce_add": (lambda d, i: bmm.box_reduce_add(d, i, (4, 4), (0, 0), "f32"),
                       [BOX, empty(torch.float32, 1, 4, 4)]),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_runs_where_its_tensors_are(gpus, name, device):
    """On the tensors' GPU and its current stream, whichever GPU is current; the
    outputs are there too, and the current GPU stays what it was."""
    call, tensors = CALLS[name]
    out = call(*(t(device) for t in tensors))
    assert [l[1:] for l in gpus.launches] == [(device, 1000 + device)]
    assert gpus.state.device == 0
    for t in out if isinstance(out, tuple) else (out,):
        if isinstance(t, torch.Tensor):
            assert t.get_device() == device


@pytest.mark.parametrize("name", [n for n, (_, ts) in CALLS.items() if len(ts) > 1])
def test_refuses_tensors_of_two_gpus(gpus, name):
    """Any one tensor on another GPU than the rest."""
    call, tensors = CALLS[name]
    for odd in range(len(tensors)):
        with pytest.raises(ValueError, match="one GPU"):
            call(*(t(int(i == odd)) for i, t in enumerate(tensors)))
    assert not gpus.launches


def test_refuses_codes_and_scales_of_two_gpus(gpus):
    q, w = XQ(0), WQ(0)
    apart = q._replace(scales=XQ(1).scales)
    for call in (lambda: bmm.mx4_dequantize(apart), lambda: bmm.mx4_mma(apart, w),
                 lambda: bmm.mx4_gated(apart, w, w)):
        with pytest.raises(ValueError, match="one GPU"):
            call()
    assert not gpus.launches
