"""The feed-forward half's calls of the Python binding on the host: stand-ins for device tensors,
streams and the library show which arguments a call hands on, and that it refuses the others before
anything reaches the GPU."""

import pytest
import torch

import grouped_nvfp4_w4a16_amd as pkg
from test_fp8_binding import BIG, Library, Stream, Tensor

F8, BF16, F32, I32, I8 = (torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32,
                          torch.int8)


class Few(Library):
    def moe_few_workspace_bytes(self, *args):
        return 1024

    def moe_shared_expert_int8_workspace_bytes(self, *args):
        return 1024


@pytest.fixture
def lib(monkeypatch):
    lib = Few()
    monkeypatch.setattr(pkg, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x55, raising=False)
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None: Tensor(shape, dtype))
    return lib


class Table:
    """An ExpertTable's fields."""

    def __init__(self, experts, n, k, device=0):
        self.n, self.k, self.num_experts = n, k, experts
        self.packed_ptrs = Tensor((experts,), torch.int64, device=device)
        self.scale_ptrs = Tensor((experts,), torch.int64, device=device)
        self.scale2 = Tensor((experts,), F32, device=device)
        self.present = [True] * experts


class Args(dict):
    """A call's tensors by name, each of which a test may replace."""

    def put(self, **kw):
        return Args({**self, **kw})


def norm_args(rows=4, cols=256):
    m = lambda dtype, c=cols: Tensor((rows, c), dtype)
    return {
        "moe_rmsnorm_bf16": Args(x=m(BF16), weight=Tensor((cols,), BF16), y=m(BF16),
                                 residual=m(BF16), h=m(BF16)),
        "moe_rmsnorm_fp8": Args(x=m(BF16), weight=Tensor((cols,), BF16), q=m(F8),
                                scale=m(F32, -(-cols // 128)), residual=m(BF16), h=m(BF16),
                                y=m(BF16)),
        "moe_rmsnorm_int8": Args(x=m(BF16), weight=Tensor((cols,), BF16), q=m(I8),
                                 scale=Tensor((rows,), F32), residual=m(BF16), h=m(BF16),
                                 y=m(BF16)),
        "moe_quant_int8": Args(x=m(BF16), q=m(I8), scale=Tensor((rows,), F32)),
    }


def gemm_args(m=4, n=144, k=256):
    a = dict(a=Tensor((m, k), I8), a_scale=Tensor((m,), F32))
    w = lambda: Tensor((n, k), I8)
    s = lambda: Tensor((n,), F32)
    return {
        "moe_dense_gemm_int8": Args(**a, b=w(), b_scale=s(), c=Tensor((m, n), BF16)),
        "moe_dense_gate_up_swiglu_int8": Args(**a, gate_w=w(), gate_scale=s(), up_w=w(),
                                              up_scale=s(), act=Tensor((m, n), BF16), limit=7.0),
    }


def few_args(rows=4, e=3, hidden=256, mi=192, top_k=2):
    common = dict(x=Tensor((rows, hidden), BF16), gate_up=Table(e, 2 * mi, hidden),
                  down=Table(e, hidden, mi), limit=7.0, out=Tensor((rows, hidden), BF16),
                  shared=Tensor((rows, hidden), BF16), ws=pkg.FewWorkspace(max(rows, 1), top_k, mi))
    ids, wts = Tensor((rows, top_k), I32), Tensor((rows, top_k), F32)
    return {
        "moe_layer_few": Args(**common, topk_ids=ids, topk_weights=wts),
        "moe_layer_few_from_logits": Args(**common, logits=Tensor((rows, e), F32), top_k=top_k,
                                          bias=Tensor((e,), F32), topk_ids=ids, topk_weights=wts),
    }


NAMES = ["moe_rmsnorm_bf16", "moe_rmsnorm_fp8", "moe_rmsnorm_int8", "moe_quant_int8",
         "moe_dense_gemm_int8", "moe_dense_gate_up_swiglu_int8", "moe_layer_few",
         "moe_layer_few_from_logits"]


def args_of(name):
    for f in (norm_args, gemm_args, few_args):
        if name in f():
            return f()[name]


def moved(t, device):
    return Tensor(t.shape, t.dtype, t.strides, device)


@pytest.mark.parametrize("name", NAMES)
def test_the_stream_of_a_call(lib, name):
    """The current device's current stream, or the given one; another device's is refused."""
    call, args = getattr(pkg, name), args_of(name)
    call(**args)
    call(**args, stream=Stream(0))
    assert [a[-1] for _, a in lib.calls] == [0x55, 0x77]
    with pytest.raises(ValueError, match="stream"):
        call(**args, stream=Stream(1))
    assert len(lib.calls) == 2


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device_launch_nothing(lib, name):
    args = args_of(name)
    for key, t in args.items():
        if isinstance(t, Tensor):
            other = moved(t, 1)
        elif isinstance(t, Table):
            other = Table(t.num_experts, t.n, t.k, 1)
        elif key == "ws":
            other = pkg.FewWorkspace(4, 2, 192)
            other.buffer = Tensor((1024,), torch.uint8, device=1)
        else:
            continue
        with pytest.raises(ValueError, match="cuda:1"):
            getattr(pkg, name)(**args.put(**{key: other}))
    assert lib.calls == []


@pytest.mark.parametrize("name", NAMES)
def test_other_types_and_shapes_are_refused(lib, name):
    """Every tensor in another type, with a row or element less, and with columns apart."""
    call, args = getattr(pkg, name), args_of(name)
    for key, t in args.items():
        if not isinstance(t, Tensor):
            continue
        with pytest.raises((TypeError, ValueError)):
            call(**args.put(**{key: Tensor(t.shape, torch.float64)}))
        with pytest.raises(ValueError):
            call(**args.put(**{key: Tensor((t.shape[0] - 1, *t.shape[1:]), t.dtype)}))
        apart = tuple(2 * s for s in t.strides)
        with pytest.raises((TypeError, ValueError)):
            call(**args.put(**{key: Tensor(t.shape, t.dtype, apart)}))
        with pytest.raises((TypeError, ValueError)):
            call(**args.put(**{key: Tensor((*t.shape, 1), t.dtype)}))
    assert lib.calls == []


@pytest.mark.parametrize("make,names", [
    (lambda: norm_args(rows=BIG), ["moe_rmsnorm_bf16", "moe_rmsnorm_fp8", "moe_rmsnorm_int8",
                                   "moe_quant_int8"]),
    (lambda: norm_args(cols=BIG), ["moe_rmsnorm_bf16", "moe_rmsnorm_fp8", "moe_rmsnorm_int8",
                                   "moe_quant_int8"]),
    (lambda: gemm_args(m=BIG), ["moe_dense_gemm_int8", "moe_dense_gate_up_swiglu_int8"]),
    (lambda: gemm_args(n=BIG), ["moe_dense_gemm_int8", "moe_dense_gate_up_swiglu_int8"]),
    (lambda: gemm_args(k=BIG), ["moe_dense_gemm_int8", "moe_dense_gate_up_swiglu_int8"])])
def test_sizes_past_32_bits_are_refused(lib, make, names):
    """The library takes 32-bit sizes: a longer one must not be cut to its low bits."""
    for name in names:
        with pytest.raises(ValueError, match="32-bit"):
            getattr(pkg, name)(**make()[name])
    assert lib.calls == []


def test_makers_refuse_sizes_past_32_bits(lib):
    with pytest.raises(ValueError, match="32-bit"):
        pkg.FewWorkspace(4, 2, BIG)
    for inter, hidden, rows in ((BIG, 64, 4), (64, BIG, 4), (64, 64, BIG)):
        w, d = Tensor((inter, hidden), I8), Tensor((hidden, inter), I8)
        s, sd = Tensor((inter,), F32), Tensor((hidden,), F32)
        with pytest.raises(ValueError, match="32-bit"):
            pkg.SharedExpertInt8(w, s, w, s, d, sd, rows)


@pytest.mark.parametrize("rows,top_k", [(0, 1), (17, 1), (-BIG, 2), (4, 65), (16, 17), (1, 257),
                                        (1, 0), (1, BIG)])
def test_a_few_workspaces_limits(lib, rows, top_k):
    with pytest.raises(ValueError):
        pkg.FewWorkspace(rows, top_k, 192)


@pytest.mark.parametrize("stride", [(1, 1), (0, 1), (258, 1), (1 << 25, 1)])
def test_a_single_rows_stride_says_nothing(lib, stride):
    """One row of a matrix of any stride: where its rows would go on does not matter."""
    for make in (norm_args, gemm_args, few_args):
        for name, args in make(1).items():
            one = {key: Tensor(t.shape, t.dtype, stride) for key, t in args.items()
                   if isinstance(t, Tensor) and len(t.shape) == 2 and t.shape[0] == 1
                   and key not in ("topk_ids", "topk_weights")}
            getattr(pkg, name)(**args.put(**one))
    calls = dict(lib.calls)
    assert calls["moe_rmsnorm_bf16"][1] == calls["moe_rmsnorm_bf16"][3] == 256
    assert calls["moe_rmsnorm_int8"][11] == calls["moe_quant_int8"][3] == 256
    assert calls["moe_dense_gemm_int8"][1] == 256 and calls["moe_dense_gemm_int8"][7] == 144
    assert calls["moe_w4a16_layer_few"][1] == 256 and calls["moe_w4a16_layer_few"][3] == 3


@pytest.mark.parametrize("stride", [0, 2])
def test_logits_rows_that_overlap_are_refused(lib, stride):
    """Rows of one set of logits expanded to many have no stride of their own."""
    args = few_args()["moe_layer_few_from_logits"]
    with pytest.raises(ValueError, match="overlap"):
        pkg.moe_layer_few_from_logits(**args.put(logits=Tensor((4, 3), F32, (stride, 1))))
    assert lib.calls == []
    pkg.moe_layer_few_from_logits(**args.put(logits=Tensor((4, 3), F32, (5, 1))))
    assert lib.calls[0][1][3] == 5


def test_a_few_layers_tables_and_workspace_fit_the_call(lib):
    args = few_args()["moe_layer_few"]
    for kw in (dict(ws=pkg.FewWorkspace(3, 2, 192)), dict(ws=pkg.FewWorkspace(4, 3, 192)),
               dict(ws=pkg.FewWorkspace(4, 2, 256)), dict(gate_up=Table(2, 384, 256)),
               dict(gate_up=Table(3, 256, 256)), dict(down=Table(3, 320, 192))):
        with pytest.raises(ValueError):
            pkg.moe_layer_few(**args.put(**kw))
    assert lib.calls == []


def shared_int8(rows=4, hidden=256, inter=192):
    w = lambda: Tensor((inter, hidden), I8)
    s = lambda: Tensor((inter,), F32)
    return pkg.SharedExpertInt8(w(), s(), w(), s(), Tensor((hidden, inter), I8),
                                Tensor((hidden,), F32), rows)


def test_the_int8_shared_expert_refuses_what_does_not_fit(lib):
    hidden, inter = 256, 192
    w = lambda **kw: Tensor((inter, hidden), I8, **kw)
    s = lambda **kw: Tensor((inter,), F32, **kw)
    d, ds = Tensor((hidden, inter), I8), Tensor((hidden,), F32)
    for bad in ((w(), s(), w(stride=(512, 1)), s(), d, ds), (w(), s(), w(), s(), w(), ds),
                (w(), ds, w(), s(), d, s()), (w(), s(device=1), w(), s(), d, ds),
                (w(), s(), w(), s(), moved(d, 1), ds)):
        with pytest.raises(ValueError):
            pkg.SharedExpertInt8(*bad, 4)
    expert = shared_int8()
    expert.out = Table(1, 1, 1)  # never reached
    expert.out.shape = (4, hidden)
    for x, xs in ((Tensor((5, hidden), I8), Tensor((5,), F32)),
                  (Tensor((4, 128), I8), Tensor((4,), F32)),
                  (Tensor((4, hidden), I8), Tensor((3,), F32)),
                  (Tensor((4, hidden), I8, (512, 2)), Tensor((4,), F32))):
        with pytest.raises(ValueError):
            expert(x, xs, 7.0)
    with pytest.raises(TypeError):
        expert(Tensor((4, hidden), BF16), Tensor((4,), F32), 7.0)
    assert lib.calls == []
