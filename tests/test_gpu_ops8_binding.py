"""The binding's check of a tensor's type against the type code beside it. Nothing is launched."""
import numpy as np
import pytest
import torch

from speculative_tree_verify_mla_b200 import kdv
from tests.test_ops8_host import attn_params, logits_params, rope_params, write_params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("make,field,code", [
    (rope_params, "x", "x_dtype"), (rope_params, "y", "y_dtype"), (write_params, "c", "dtype"), (write_params, "k_rope", "dtype"),
    (attn_params, "q", "dtype"), (attn_params, "o", "out_dtype"), (logits_params, "logits", "dtype"), (logits_params, "out", "out_dtype")])
def test_types_and_their_codes(make, field, code):
    t = {kdv.KDV_BF16: torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), kdv.KDV_F32: torch.zeros(4, 64, device="cuda")}
    for a in t:
        for b in t:
            if a == b:
                assert getattr(make(**{field: t[a], code: b}), field) == t[a].data_ptr()
            else:
                with pytest.raises(TypeError, match=code):
                    make(**{field: t[a], code: b})
    with pytest.raises(TypeError, match="unsupported"):
        make(**{field: torch.zeros(4, dtype=torch.float16, device="cuda")})


def test_a_code_that_is_not_given_is_bf16():
    with pytest.raises(TypeError):
        kdv.make_rope_params(x=torch.zeros(4, device="cuda"))
    kdv.make_rope_params(x=torch.zeros(4, dtype=torch.bfloat16, device="cuda"), h_inv_freq=np.ones(1))
