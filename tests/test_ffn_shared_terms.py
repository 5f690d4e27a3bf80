"""What a few-token layer takes as its shared term, on the host."""

import pytest

import grouped_nvfp4_w4a16_amd as pkg
from test_ffn_binding import BF16, F32, I8, Tensor, few_args, lib, shared_int8  # noqa: F401
from test_fp8_binding import Partials


class Fp8(pkg.SharedExpertFp8):
    def __init__(self):
        self.out = Tensor((4, 256), BF16)


@pytest.mark.parametrize("name", ["moe_layer_few", "moe_layer_few_from_logits"])
def test_terms_of_other_kinds_are_refused_before_a_launch(lib, name):  # noqa: F811
    args = few_args()[name]
    for term in (Partials(0), Fp8(), object(), 1.0, Tensor((4, 256), F32)):
        with pytest.raises(TypeError, match="shared"):
            getattr(pkg, name)(**args.put(shared=term))
    with pytest.raises(ValueError, match="shared"):
        getattr(pkg, name)(**args.put(shared=Tensor((4, 512), BF16)))
    assert lib.calls == []


def test_an_int8_expert_runs_before_the_layer(lib, monkeypatch):  # noqa: F811
    # as much of torch's slicing as the expert needs of its buffers
    monkeypatch.setattr(Tensor, "__getitem__", lambda t, s: Tensor((s.stop, *t.shape[1:]), t.dtype),
                        raising=False)
    pkg.moe_layer_few(**few_args()["moe_layer_few"].put(shared=shared_int8()))
    assert [n for n, _ in lib.calls] == ["moe_quant_int8", "moe_shared_expert_int8",
                                         "moe_w4a16_layer_few"]
    with pytest.raises(ValueError, match="rows"):
        pkg.moe_layer_few(**few_args()["moe_layer_few"].put(shared=shared_int8(rows=3)))
    assert len(lib.calls) == 3
