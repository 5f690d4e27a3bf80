"""The FP8 calls of the Python binding on the host: stand-ins for device tensors, streams and
the library show which arguments a call hands on, and that it refuses the others before
anything reaches the GPU."""

import contextlib

import pytest
import torch

import grouped_nvfp4_w4a16_amd as pkg

F8, BF16, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32


class Tensor:
    """As much of a device tensor as the binding asks for; it holds no memory."""

    is_cuda = True

    def __init__(self, shape, dtype, stride=None, device=0, ptr=0x10000):
        self.shape, self.dtype, self.index, self.ptr = torch.Size(shape), dtype, device, ptr
        dense, n = [], 1
        for d in reversed(self.shape):
            dense.insert(0, n)
            n *= d
        self.strides = tuple(dense) if stride is None else tuple(stride)
        self.dense = self.strides == tuple(dense)

    def stride(self, dim=None):
        return self.strides if dim is None else self.strides[dim]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return self.dense

    def get_device(self):
        return self.index

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def data_ptr(self):
        return self.ptr


class Library:
    """Records every call's arguments; each succeeds."""

    def __init__(self):
        self.calls = []

    def moe_fp8_swiglu_workspace_bytes(self, *args):
        return 0

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class Table:
    """An Fp8ExpertTable's fields."""

    def __init__(self, experts, n, k, gate_up=False, device=0):
        self.n, self.k, self.num_experts, self.gate_up = n, k, experts, gate_up
        self.present = [True] * experts
        self.weight_ptrs = Tensor((experts,), torch.int64, device=device)
        self.scale_ptrs = Tensor((experts,), torch.int64, device=device)


class Stream:
    def __init__(self, device_index, handle=0x77):
        self.device_index, self.cuda_stream = device_index, handle


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(pkg, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x55, raising=False)
    return lib


def _quant(rows=4, cols=256, **kw):
    pkg.moe_quant_fp8(Tensor((rows, cols), BF16), Tensor((rows, cols), F8),
                      Tensor((rows, -(-cols // 128)), F32), **kw)


def _dense(m=4, n=144, k=256, **kw):
    pkg.moe_dense_gemm_fp8(Tensor((m, k), F8), Tensor((m, 2), F32), Tensor((n, k), F8),
                           Tensor((-(-n // 128), 2), F32), Tensor((m, n), BF16), **kw)


def _dense_swiglu(m=4, n=144, k=256, **kw):
    w, s = Tensor((n, k), F8), Tensor((2, 2), F32)
    pkg.moe_dense_gate_up_swiglu_fp8(Tensor((m, k), F8), Tensor((m, 2), F32), w, s, w, s,
                                     Tensor((m, n), F8), Tensor((m, 2), F32), 7.0, **kw)


def _grouped(rows=4, **kw):
    pkg.moe_w8a8_grouped_gemm(Tensor((rows, 256), F8), Tensor((rows, 2), F32), Table(3, 144, 256),
                              Tensor((4,), I32), Tensor((rows, 144), BF16), **kw)


def _grouped_swiglu(rows=4, **kw):
    pkg.moe_w8a8_grouped_gemm_swiglu(Tensor((rows, 256), F8), Tensor((rows, 2), F32),
                                     Table(3, 288, 256, True), Tensor((4,), I32),
                                     Tensor((rows, 144), F8), Tensor((rows, 2), F32), 7.0, **kw)


CALLS = {"moe_quant_fp8": _quant, "moe_dense_gemm_fp8": _dense,
         "moe_dense_gate_up_swiglu_fp8": _dense_swiglu, "moe_w8a8_grouped_gemm": _grouped,
         "moe_w8a8_grouped_gemm_swiglu": _grouped_swiglu}


@pytest.mark.parametrize("name", CALLS)
def test_the_stream_of_a_call(lib, name):
    """The current device's current stream, or the given one; a stream of another device would
    run a kernel prepared for the current one, on memory of the current one: refused."""
    CALLS[name]()
    CALLS[name](stream=Stream(0))
    assert [(n, a[-1]) for n, a in lib.calls] == [(name, 0x55), (name, 0x77)]
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](stream=Stream(1))
    assert len(lib.calls) == 2


class Workspace:
    """An Fp8Workspace's fields for 4 rows, top 2 of 3 experts, hidden 256, width 144."""

    max_rows, top_k, num_experts, hidden, moe_intermediate = 4, 2, 3, 256, 144

    def __init__(self, device=0):
        self.x = Tensor((4, 256), F8, device=device)


class Shared:
    """A shared expert's output buffer."""

    def __init__(self, device):
        self.out = Tensor((4, 256), BF16, device=device)


class Partials(pkg.SharedPartials):
    def __init__(self, device):
        self.partials, self.ways = Tensor((2, 4, 256), F32, device=device), 2


@pytest.mark.parametrize("case", ["stream", "x", "workspace", "gate_up", "down", "shared term",
                                  "shared partials", "shared expert"])
def test_a_layer_on_another_device_launches_nothing(lib, case):
    at = {case: 1}
    ids, w = Tensor((4, 2), I32), Tensor((4, 2), F32)
    shared = {"shared term": Tensor((4, 256), BF16, device=1), "shared partials": Partials(1),
              "shared expert": Shared(1)}.get(case)
    with pytest.raises(ValueError, match="cuda:1"):
        pkg.moe_layer_fp8(Tensor((4, 256), BF16, device=at.get("x", 0)), ids, w,
                          Table(3, 288, 256, True, at.get("gate_up", 0)),
                          Table(3, 256, 144, device=at.get("down", 0)), 7.0,
                          Workspace(at.get("workspace", 0)), Tensor((4, 256), BF16), shared,
                          stream=Stream(at.get("stream", 0)))
    assert lib.calls == []


BIG = 2 ** 32 + 16  # 16 in 32 bits


@pytest.mark.parametrize("call", [
    lambda: _quant(rows=BIG, cols=16), lambda: _quant(rows=1, cols=BIG), lambda: _dense(m=BIG),
    lambda: _dense(n=BIG), lambda: _dense_swiglu(m=BIG), lambda: _grouped(rows=BIG),
    lambda: _grouped_swiglu(rows=BIG), lambda: _grouped(max_rows=-BIG),
    lambda: pkg.moe_fp8_swiglu_workspace_bytes(BIG, 0, 2048, 6144),
    lambda: pkg.moe_fp8_swiglu_workspace_bytes(8, 0, BIG, 6144)])
def test_sizes_past_32_bits_are_refused(lib, call):
    """The library takes 32-bit sizes: a longer one must not be cut to its low bits."""
    with pytest.raises(ValueError, match="32-bit"):
        call()
    assert lib.calls == []


def test_gathered_rows_past_32_bits_are_refused(lib):
    for grouped, table, out in ((pkg.moe_w8a8_grouped_gemm, Table(3, 144, 256), BF16),
                                (pkg.moe_w8a8_grouped_gemm_swiglu, Table(3, 288, 256, True), F8)):
        rest = () if out is BF16 else (Tensor((4, 2), F32), 7.0)
        with pytest.raises(ValueError, match="32-bit"):
            grouped(Tensor((BIG, 256), F8), Tensor((BIG, 2), F32), table, Tensor((4,), I32),
                    Tensor((4, 144), out), *rest, a_gather=Tensor((4,), I32))
    assert lib.calls == []


@pytest.mark.parametrize("stride", [(1, 1), (0, 1), (258, 1), (1 << 23, 1)])
def test_a_single_rows_stride_says_nothing(lib, stride):
    """One row of a matrix of any stride (odd, zero, past 2^22): where its rows would go on does
    not matter."""
    def row(cols, dtype):
        return Tensor((1, cols), dtype, stride)

    one = Tensor((1, 2), F32, stride)
    pkg.moe_quant_fp8(row(256, BF16), row(256, F8), one)
    pkg.moe_dense_gemm_fp8(row(256, F8), one, Tensor((144, 256), F8), Tensor((2, 2), F32),
                           row(144, BF16))
    w, s = Tensor((144, 256), F8), Tensor((2, 2), F32)
    pkg.moe_dense_gate_up_swiglu_fp8(row(256, F8), one, w, s, w, s, row(144, F8), one, 7.0)
    off = Tensor((4,), I32)
    pkg.moe_w8a8_grouped_gemm(row(250, F8), one, Table(3, 144, 240), off, row(144, BF16))
    pkg.moe_w8a8_grouped_gemm_swiglu(row(256, F8), one, Table(3, 288, 256, True), off,
                                     row(144, F8), one, 7.0)
    lds = {name: args for name, args in lib.calls}
    assert lds["moe_quant_fp8"][1] == lds["moe_quant_fp8"][3] == 256
    assert lds["moe_dense_gemm_fp8"][1] == 256 and lds["moe_dense_gemm_fp8"][8] == 144
    assert lds["moe_dense_gate_up_swiglu_fp8"][1] == 256
    assert lds["moe_dense_gate_up_swiglu_fp8"][10] == 144
    assert lds["moe_w8a8_grouped_gemm"][1] == 256 and lds["moe_w8a8_grouped_gemm"][11] == 144
    assert lds["moe_w8a8_grouped_gemm_swiglu"][11] == 144
    assert lds["moe_quant_fp8"][5] == lds["moe_dense_gemm_fp8"][3] == 2
    # of two rows it is what it is
    pkg.moe_quant_fp8(Tensor((2, 256), BF16, (264, 1)), Tensor((2, 256), F8, (272, 1)),
                      Tensor((2, 2), F32))
    assert lib.calls[-1][1][1] == 264 and lib.calls[-1][1][3] == 272


@pytest.mark.parametrize("rows", [0, 1, 4])
def test_quantising_no_columns_does_nothing(lib, rows):
    """A matrix without columns has no stride to speak of (torch gives 1)."""
    empty = torch.empty(rows, 0)
    pkg.moe_quant_fp8(Tensor((rows, 0), BF16, empty.stride()), Tensor((rows, 0), F8, empty.stride()),
                      Tensor((rows, 0), F32, empty.stride()))
    for _, args in lib.calls:
        assert args[1] % 8 == 0 and args[3] % 16 == 0


class Sized(Library):
    """A library whose split workspace is largest in the middle of the row counts."""

    def moe_fp8_swiglu_workspace_bytes(self, rows, experts, width, k):
        return {0: 256, 1: 512}.get(abs(rows - (8 if experts else 4)), 0)


def test_the_layer_holds_its_split_workspaces(monkeypatch):
    """The largest need over every row count up to max_rows, which the last one may not be;
    none where no row count splits."""
    monkeypatch.setattr(pkg, "load", Sized)
    monkeypatch.setattr(pkg, "_split_device", lambda device: contextlib.nullcontext())
    assert pkg.Fp8Workspace(6, 2, 3, 256, 144, device="cpu").split.numel() == 256
    assert pkg.Fp8Workspace(6, 3, 3, 256, 144, device="cpu").split.numel() == 512
    assert pkg.Fp8Workspace(2, 2, 3, 256, 144, device="cpu").split is None
    assert pkg.Fp8Workspace(2, 0, 3, 256, 144, device="cpu").split is None
    w, s = torch.empty(144, 256), torch.empty(2, 2)
    for rows, need in ((9, 512), (3, 512), (1, None)):
        sh = pkg.SharedExpertFp8(w, s, w, s, w.t().contiguous(), s, rows)
        assert (None if sh.split is None else sh.split.numel()) == need


def test_the_current_stream_without_torchs_short_cut(lib, monkeypatch):
    """torch's internal query is a short cut: without it the public one serves."""
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(0, 0x99))
    for name, call in CALLS.items():
        call()
        assert lib.calls[-1][0] == name and lib.calls[-1][1][-1] == 0x99
    with pytest.raises(ValueError, match="cuda:1"):
        _quant(stream=Stream(1))
