"""The comparisons of the expert-layer operators' bf16 results once more, with
results that have to be numbers: rows without a pair hold NaN and must not be
read, and a NaN that leaks into a result is refused (strict_reference)."""
import pytest

import expert_reference
import strict_reference
import train_reference
from test_gpu_experts import (test_a_layer_end_to_end, test_expert_gemm, test_layer_fused,  # noqa: F401
                              test_products_do_not_depend_on_when_loads_arrive, test_rmsnorm)
from test_gpu_train import (_gpu, test_activation_backward, test_activation_backward_far_values,  # noqa: F401
                            test_combine_backward, test_gated, test_grad_input, test_grad_weight, test_grad_weight_splits_rows,
                            test_linear, test_most_experts)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _strict(monkeypatch):
    monkeypatch.setattr(expert_reference, "assert_bf16", strict_reference.assert_bf16)
    monkeypatch.setattr(train_reference, "assert_bf16", strict_reference.assert_bf16)
